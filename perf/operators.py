"""Cases of the training operators that stand beside the row norms: group norm with an activation over channels-last
tensors, forward (``gn_fwd``) and backward (``gn_bwd``), the global norm of a list of gradients (``grad_norm``) and
clipping by it (``grad_clip``).

A group norm case gives the batch, the spatial positions (height x width, or frames), the channels and the groups; x and
dy are [batch, positions, channels]. A gradient case gives the layers and the width of a network and which of its
gradients are in the list:
  block     per layer four [width, width] projections, [4 width, width] and [width, 4 width], and two [width] norm weights
  adapters  per layer a [rank, width] and a [width, rank] factor
  vectors   per layer the two [width] column gradients of a norm
``flat`` gradients are views of one buffer, one after the other, so they start at any element. In a ``mixed`` list vectors
are float32 and matrices bfloat16.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
MAX_NORM = 1.0


def _gn(name, op, dtype, batch, positions, channels, groups, act):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "positions": positions, "channels": channels,
            "groups": groups, "act": act}


def _gr(name, op, dtype, kind, layers, width, rank=0, flat=False):
    return {"name": name, "op": op, "dtype": dtype, "kind": kind, "layers": layers, "width": width, "rank": rank,
            "flat": flat}


def listed():
    return [
        # the lowest resolution of an image network, one image: latency
        _gn("gn_fwd_bf16_1x64x1280", "gn_fwd", "bf16", 1, 8 * 8, 1280, 32, "silu"),
        # the highest resolution of a latent image network, two images; ten channels a group
        _gn("gn_fwd_bf16_2x4096x320", "gn_fwd", "bf16", 2, 64 * 64, 320, 32, "silu"),
        # odd positions, six channels a group, norm alone
        _gn("gn_fwd_f32_3x1517x180", "gn_fwd", "f32", 3, 37 * 41, 180, 30, "none"),
        # the last stage of an image decoder: one image larger than the cache
        _gn("gn_fwd_bf16_1x262144x256", "gn_fwd", "bf16", 1, 512 * 512, 256, 32, "silu"),
        # training at a low resolution
        _gn("gn_bwd_bf16_2x256x1280", "gn_bwd", "bf16", 2, 16 * 16, 1280, 32, "silu"),
        # training at a latent image network's highest resolution
        _gn("gn_bwd_f16_8x4096x320", "gn_bwd", "f16", 8, 64 * 64, 320, 32, "silu"),
        # odd positions, six channels a group
        _gn("gn_bwd_f32_3x1517x180", "gn_bwd", "f32", 3, 37 * 41, 180, 30, "gelu"),
        # training an image decoder's stage on a batch
        _gn("gn_bwd_bf16_4x65536x256", "gn_bwd", "bf16", 4, 256 * 256, 256, 32, "silu"),
        # the column gradients of 12 norms, as the row norms' backward writes them: latency
        _gr("grad_norm_f32_vectors", "grad_norm", "f32", "vectors", 12, 1024),
        # a network of 0.8 G parameters
        _gr("grad_norm_bf16_block", "grad_norm", "bf16", "block", 16, 2048),
        # low-rank adapters in one flat buffer, odd sizes
        _gr("grad_clip_mixed_adapters", "grad_clip", "mixed", "adapters", 24, 5001, 9, True),
        # a quarter of a G of float32 gradients
        _gr("grad_clip_f32_block", "grad_clip", "f32", "block", 5, 2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "grad_norm", "grad_clip"])
    if op.startswith("gn"):
        per_group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 20, 24, 32, 40, 64])
        groups = rng.choice([1, 4, 8, 16, 25, 32, 32, 32, 64])
        channels = per_group * groups
        batch = _log_int(rng, 1, 16)
        least = max(64 * batch * channels, 1 << 13)
        values = _log_int(rng, least, 1 << 26)
        return {"op": op, "dtype": rng.choice(list(DTYPES)), "batch": batch,
                "positions": max(64, values // (batch * channels)), "channels": channels, "groups": groups,
                "act": rng.choice(["none", "silu", "gelu"])}
    kind = rng.choice(["block", "adapters", "vectors"])
    if kind == "vectors":
        layers, width, rank = rng.randint(1, 30), _log_int(rng, 16, 65536), 0
    elif kind == "adapters":
        layers, width, rank = rng.randint(1, 30), _log_int(rng, 64, 16384), _log_int(rng, 1, 128)
    else:
        width, rank = _log_int(rng, 64, 2048), 0
        layers = rng.randint(1, 5 if op == "grad_clip" else 16)
    return {"op": op, "dtype": rng.choice(["f32", "bf16", "f16", "mixed"]), "kind": kind, "layers": layers,
            "width": width, "rank": rank, "flat": rng.choice([False, True])}


def _shapes(case):
    w, r = case["width"], case["rank"]
    layer = {"block": [(w, w)] * 4 + [(4 * w, w), (w, 4 * w), (w,), (w,)],
             "adapters": [(r, w), (w, r)],
             "vectors": [(w,), (w,)]}[case["kind"]]
    return layer * case["layers"]


def _dtype_of(case, shape):
    if case["dtype"] == "mixed":
        return torch.float32 if len(shape) == 1 or case["kind"] == "adapters" and shape[0] < shape[1] else torch.bfloat16
    return DTYPES[case["dtype"]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"].startswith("gn"):
        b, s, c, n = case["batch"], case["positions"], case["channels"], case["groups"]
        dt = DTYPES[case["dtype"]]
        # channels of a convolution's output: each with an offset and a scale of its own
        x = normal(b, s, c).mul_(0.5 + torch.rand(c, generator=g, device="cuda")).add_(0.5 * normal(c)).to(dt)
        state = {"case": case, "x": x, "gamma": (1 + 0.1 * normal(c)).to(dt), "beta": (0.1 * normal(c)).to(dt)}
        if case["op"] == "gn_bwd":
            state["dy"] = normal(b, s, c).to(dt)
            # the statistics that the forward call saved
            sums = x.sum(1, dtype=torch.float64).view(b, n, -1).sum(2)
            mean = sums / (s * c // n)
            var = torch.stack([(x[i].float() - mean[i].float().repeat_interleave(c // n)).square().sum(0, dtype=torch.float64)
                               for i in range(b)]).view(b, n, -1).sum(2) / (s * c // n)
            state["mean"], state["rstd"] = mean.float(), (var + EPS).rsqrt().float()
        return state

    shapes = _shapes(case)
    # gradients of different tensors differ in scale by a factor of a hundred
    scales = [10.0 ** (-4 + 2 * v) for v in torch.rand(len(shapes), generator=torch.Generator().manual_seed(seed)).tolist()]
    if case["flat"]:
        buffers = {}
        for dt in {_dtype_of(case, s) for s in shapes}:
            buffers[dt] = torch.empty(sum(math.prod(s) for s in shapes if _dtype_of(case, s) == dt), dtype=dt, device="cuda")
        grads, at = [], dict.fromkeys(buffers, 0)
        for s, a in zip(shapes, scales):
            dt = _dtype_of(case, s)
            grads.append(buffers[dt][at[dt]:at[dt] + math.prod(s)].view(s).copy_(normal(*s) * a))
            at[dt] += math.prod(s)
    else:
        grads = [(normal(*s) * a).to(_dtype_of(case, s)) for s, a in zip(shapes, scales)]
    state = {"case": case, "grads": grads}
    if case["op"] == "grad_clip":  # the clipped gradients go to buffers of their own: every pass then has the same inputs
        state["out"] = [torch.empty_like(t) for t in grads]
    return state


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _gn_fwd_plain(state):
    case = state["case"]
    b, s, c, n = case["batch"], case["positions"], case["channels"], case["groups"]
    x = state["x"].float().view(b, s, n, c // n)
    mean = x.mean((1, 3), keepdim=True)
    x = x - mean
    rstd = 1 / torch.sqrt(x.square().mean((1, 3), keepdim=True) + EPS)
    z = (x * rstd).view(b, s, c) * state["gamma"].float() + state["beta"].float()
    return _act(z, case["act"]).to(state["x"].dtype), mean.view(b, n), rstd.view(b, n)


def _gn_bwd_plain(state):
    case = state["case"]
    b, s, c, n = case["batch"], case["positions"], case["channels"], case["groups"]
    gamma = state["gamma"].float()
    rstd = state["rstd"].view(b, 1, n, 1)
    xhat = ((state["x"].float().view(b, s, n, c // n) - state["mean"].view(b, 1, n, 1)) * rstd).view(b, s, c)
    dz = state["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_slope(xhat * gamma + state["beta"].float(), case["act"])
    dgamma, dbeta = (dz * xhat).sum((0, 1)), dz.sum((0, 1))
    gr, xhat = (dz * gamma).view(b, s, n, c // n), xhat.view(b, s, n, c // n)
    dx = rstd * (gr - gr.mean((1, 3), keepdim=True) - xhat * (gr * xhat).mean((1, 3), keepdim=True))
    return dx.view(b, s, c).to(state["x"].dtype), dgamma, dbeta


def _grad_norm_plain(grads):
    # 64 bits: the sums are long, and squares of small gradients fall out of float32's range
    return torch.stack([t.double().square().sum() for t in grads]).sum().sqrt()


def _grad_clip_plain(state):
    norm = _grad_norm_plain(state["grads"])
    coef = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0).float()
    return [o.copy_(t.float() * coef) for t, o in zip(state["grads"], state["out"])], norm.float()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import row_wise_normalization_ln_gb300 as rn
        if op == "gn_fwd":
            return rn.gn_fwd(state["x"], state["gamma"], state["beta"], case["groups"], EPS, activation=case["act"])
        if op == "gn_bwd":
            return rn.gn_bwd(state["dy"], state["x"], state["gamma"], state["beta"], state["mean"], state["rstd"],
                             case["groups"], activation=case["act"])
        if op == "grad_norm":
            return rn.grad_norm(state["grads"])
        return rn.grad_clip(state["grads"], MAX_NORM, out=state["out"])
    if op == "gn_fwd":
        return _gn_fwd_plain(state)
    if op == "gn_bwd":
        return _gn_bwd_plain(state)
    if op == "grad_norm":
        return _grad_norm_plain(state["grads"]).float()
    return _grad_clip_plain(state)


def work(case):
    if case["op"].startswith("gn"):
        values = case["batch"] * case["positions"] * case["channels"]
        e = DTYPES[case["dtype"]].itemsize
        c, stats = case["channels"], 8 * case["batch"] * case["groups"]
        if case["op"] == "gn_fwd":  # x, gamma, beta in; y, mean, rstd out
            return {"bytes": 2 * values * e + 2 * c * e + stats, "flops": (8 + 4 * (case["act"] != "none")) * values}
        # dy, x, gamma, beta, mean, rstd in; dx, dgamma, dbeta out
        return {"bytes": 3 * values * e + 2 * c * e + stats + 8 * c, "flops": (14 + 8 * (case["act"] != "none")) * values}
    read = sum(math.prod(s) * _dtype_of(case, s).itemsize for s in _shapes(case))
    values = sum(math.prod(s) for s in _shapes(case))
    if case["op"] == "grad_norm":
        return {"bytes": read + 4, "flops": 2 * values}
    return {"bytes": 2 * read + 4, "flops": 3 * values}


def exact(case, seed):
    state = prepare(case, seed)
    f = torch.float64
    if case["op"].startswith("grad"):
        total = sum(float((t.to(f) * t.to(f)).sum()) for t in state["grads"])
        norm = math.sqrt(total)
        if case["op"] == "grad_norm":
            return torch.tensor(norm, dtype=f)
        coef = min(1.0, MAX_NORM / (norm + 1e-6))
        return [t.to(f) * coef for t in state["grads"]], torch.tensor(norm, dtype=f)

    n, act = case["groups"], case["act"]
    b, c = case["batch"], case["channels"]
    d = c // n
    gamma, beta = state["gamma"].to(f), state["beta"].to(f)
    outs = []
    dgamma, dbeta = torch.zeros(c, dtype=f, device="cuda"), torch.zeros(c, dtype=f, device="cuda")
    # image by image, so that the 64-bit copies stay small
    for i in range(b):
        x = state["x"][i].to(f)
        per = x.shape[0] * d
        if case["op"] == "gn_fwd":
            mu = x.sum(0).view(n, d).sum(1) / per
            xc = x - mu.repeat_interleave(d)
            r = ((xc * xc).sum(0).view(n, d).sum(1) / per + EPS) ** -0.5
            z = xc * r.repeat_interleave(d) * gamma + beta
            y = z * torch.sigmoid(z) if act == "silu" else z * torch.special.ndtr(z) if act == "gelu" else z
            outs.append((y, mu, r))
            continue
        mu, r = state["mean"][i].to(f).repeat_interleave(d), state["rstd"][i].to(f).repeat_interleave(d)
        xh, dz = (x - mu) * r, state["dy"][i].to(f)
        z = xh * gamma + beta
        if act == "silu":
            p = torch.sigmoid(z)
            dz = dz * (p + z * p * (1 - p))
        elif act == "gelu":
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        s1, s2 = dz.sum(0), (dz * xh).sum(0)
        dbeta += s1
        dgamma += s2
        m1 = ((gamma * s1).view(n, d).sum(1) / per).repeat_interleave(d)
        m2 = ((gamma * s2).view(n, d).sum(1) / per).repeat_interleave(d)
        outs.append(r * (dz * gamma - m1 - xh * m2))
    if case["op"] == "gn_fwd":
        return tuple(torch.stack([o[k] for o in outs]) for k in range(3))
    return torch.stack(outs), dgamma, dbeta
