"""Cases of the row norms inside a transformer block, beside the plain and the fused-add norms.

rope_fwd, rope_bwd  RMSNorm of every query and key head with the rotary position rotation in the same pass
                    (``rms_fwd_rope``, ``rms_bwd_rope``): queries [tokens, heads, width] and keys [tokens, kv_heads, width],
                    a weight [width] each, tables of cosines and sines [positions, rotary / 2], one position per token. The
                    first ``rotary`` values of a head rotate, as pairs (i, i + rotary / 2) or, ``interleaved``,
                    (2 i, 2 i + 1). A negative position marks a padding token: its outputs are zero.
drop_fwd, drop_bwd  dropout of a block's output, the residual add and the norm of the sum (``ln_fwd_dropout_add``,
                    ``rms_fwd_dropout_add`` and their ``_bwd_``): h = residual + x * keep / P(keep), y = norm(h). The mask
                    comes from a counter-based generator and is never stored: value e of the flattened x uses 16-bit word
                    e % 8 of Philox4x32-7 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
                    2011) with the counter (e / 8, offset) and the key seed, and is dropped where that word is below
                    round(65536 p).
add_bwd             the backward of the fused add + norm, without dropout (``ln_bwd_add``, ``rms_bwd_add``): the residual
                    stream's gradient and the norm's in one pass.
"""
import functools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def _rope(name, op, dtype, tokens, heads, kv_heads, width, rotary, interleaved, packed, positions, decode):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "width": width,
            "rotary": rotary, "interleaved": interleaved, "packed": packed, "positions": positions, "decode": decode}


def _rows(name, op, norm, dtype, rows, cols, p):
    return {"name": name, "op": op, "norm": norm, "dtype": dtype, "rows": rows, "cols": cols, "p": p}


def listed():
    return [
        # one token of one sequence being answered: latency. Eight query heads share a key head.
        _rope("rope_fwd_bf16_1x32x128", "rope_fwd", "bf16", 1, 32, 4, 128, 128, False, True, 32768, True),
        # a batch that answers, with padding tokens; narrow heads, part of each rotated in neighbouring pairs
        _rope("rope_fwd_f16_501x14x80", "rope_fwd", "f16", 501, 14, 2, 80, 32, True, True, 131072, True),
        # a training step's tokens, heads split out of the projection's output
        _rope("rope_fwd_bf16_16384x32x128", "rope_fwd", "bf16", 16384, 32, 8, 128, 128, False, True, 4096, False),
        # odd tokens, as many key as query heads, a quarter of each head rotated, separate buffers
        _rope("rope_bwd_f32_1023x12x96", "rope_bwd", "f32", 1023, 12, 12, 96, 24, False, False, 2048, False),
        # the backward of the training step's tokens, into the projection's packed gradient
        _rope("rope_bwd_bf16_16384x32x128", "rope_bwd", "bf16", 16384, 32, 8, 128, 128, False, True, 4096, False),
        # a small network's step: latency
        _rows("drop_fwd_ln_f32_128x1024", "drop_fwd", "ln", "f32", 128, 1024, 0.1),
        # rows of odd width
        _rows("drop_fwd_ln_bf16_4096x5001", "drop_fwd", "ln", "bf16", 4096, 5001, 0.1),
        # many short rows, the largest
        _rows("drop_fwd_rms_bf16_65536x2048", "drop_fwd", "rms", "bf16", 65536, 2048, 0.05),
        # a wide layer's training step
        _rows("drop_bwd_ln_bf16_4096x8192", "drop_bwd", "ln", "bf16", 4096, 8192, 0.1),
        # float32 rows, not a power of two
        _rows("drop_bwd_rms_f32_2047x5000", "drop_bwd", "rms", "f32", 2047, 5000, 0.2),
        # a small step: latency
        _rows("add_bwd_ln_f16_515x768", "add_bwd", "ln", "f16", 515, 768, 0.0),
        # a network without dropout
        _rows("add_bwd_rms_bf16_8192x4096", "add_bwd", "rms", "bf16", 8192, 4096, 0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "drop_fwd", "drop_bwd", "add_bwd"])
    dtype = rng.choice(list(DTYPES))
    size = DTYPES[dtype].itemsize
    if op.startswith("rope"):
        width = rng.choice([32, 48, 64, 64, 72, 80, 96, 100, 112, 128, 128, 128, 160, 192, 256])
        rotary = rng.choice([width, width, width, width // 4 * 2, width // 8 * 2])
        kv_heads = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        heads = min(64, kv_heads * rng.choice([1, 2, 3, 4, 7, 8]))
        # as many bytes at most as the largest of these listed
        tokens = _log_int(rng, 1, min(32768, (1 << 28) // (size * (heads + kv_heads) * width)))
        return {"op": op, "dtype": dtype, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "width": width,
                "rotary": rotary, "interleaved": rng.choice([False, True]), "packed": rng.choice([False, True]),
                "positions": _log_int(rng, 64, 131072), "decode": op == "rope_fwd" and rng.choice([False, True])}
    cols = _log_int(rng, 64, 16384)
    if rng.random() < 0.7:  # widths are mostly whole vectors
        cols = -(-cols // 8) * 8
    rows = _log_int(rng, 1, min(65536, (1 << 29) // (4 * size * cols)))
    return {"op": op, "norm": rng.choice(["ln", "rms"]), "dtype": dtype, "rows": rows, "cols": cols,
            "p": 0.0 if op == "add_bwd" else rng.choice([0.0, 0.05, 0.1, 0.1, 0.2, 0.5])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"].startswith("rope"):
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["width"]
        state = {"case": case}
        # the tables of the angles, made once in 64 bits: position * 10000^(-2 i / rotary)
        freq = 10000.0 ** (-torch.arange(0, case["rotary"], 2, dtype=torch.float64, device="cuda") / case["rotary"])
        angle = torch.arange(case["positions"], dtype=torch.float64, device="cuda")[:, None] * freq
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
        if case["decode"]:  # every token at its own sequence's end; one in eight pads the batch
            pos = torch.randint(case["positions"], (t,), generator=g, device="cuda")
            pos[torch.rand(t, generator=g, device="cuda") < 0.125] = -1
            pos[0] = case["positions"] - 1
        else:  # sequences one after the other
            length = int(torch.randint(max(1, case["positions"] // 2), case["positions"] + 1, (1,), generator=g, device="cuda"))
            pos = torch.arange(t, device="cuda") % length
        state["pos"] = pos
        state["wq"], state["wk"] = (1 + 0.2 * normal(d)).to(dt), (1 + 0.2 * normal(d)).to(dt)
        # projections: heads of different scales
        scale = torch.exp(0.5 * normal(hq + 2 * hk, 1))
        if case["packed"]:
            state["qkv"] = (normal(t, hq + 2 * hk, d) * scale).to(dt).view(t, -1)
        else:
            state["q"], state["k"] = ((normal(t, h, d) * s).to(dt) for h, s in ((hq, scale[:hq]), (hk, scale[hq:hq + hk])))
        if case["op"] == "rope_bwd":
            state["dq"], state["dk"] = normal(t, hq, d).to(dt), normal(t, hk, d).to(dt)
            if case["packed"]:
                state["dqkv"] = torch.empty_like(state["qkv"])
        return state

    m, n = case["rows"], case["cols"]
    state = {"case": case, "rng": torch.randint(1 << 40, (2,), generator=g, device="cuda")}
    if case["norm"] == "ln":
        state["gamma"], state["beta"] = (1 + 0.2 * normal(n)).to(dt), (0.1 * normal(n)).to(dt)
    else:
        state["gamma"] = (1 + 0.2 * normal(n)).to(dt)
    # the residual stream: channels with offsets and scales of their own
    stream = normal(m, n).mul_(0.5 + torch.rand(n, generator=g, device="cuda")).add_(0.5 * normal(n)).to(dt)
    if case["op"] == "drop_fwd":
        state["x"], state["residual"] = normal(m, n).to(dt), stream
        return state
    state["h"], state["dy"], state["dh"] = stream, normal(m, n).to(dt), normal(m, n).to(dt)
    if case["norm"] == "ln":  # the statistics that the forward call saved
        mean = stream.sum(1, dtype=torch.float64) / n
        var = torch.cat([(b.double() - mu[:, None]).square().mean(1) for b, mu in zip(stream.split(4096), mean.split(4096))])
        state["mean"], state["rstd"] = mean.float(), (var + EPS).rsqrt().float()
    return state


def _heads(flat, case):
    """Queries and keys in a packed [tokens, (heads + 2 kv_heads) width] buffer."""
    t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["width"]
    return flat[:, :hq * d].view(t, hq, d), flat[:, hq * d:(hq + hk) * d].view(t, hk, d)


def _rotate(x, cos, sin, case):
    r = case["rotary"]
    x, rest = x[..., :r], x[..., r:]
    if case["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), rest), -1)
    a, b = x[..., :r // 2], x[..., r // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1)


def _angles(state):
    pos = state["pos"]
    at = pos.clamp(min=0)
    return state["cos"][at][:, None], state["sin"][at][:, None], (pos >= 0).float()[:, None, None]


def _rope_fwd_plain(x, w, angles, case):
    cos, sin, on = angles
    v = x.float()
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()
    return torch.where(on > 0, _rotate(v, cos, sin, case), 0.0).to(x.dtype)


def _rope_bwd_plain(dy, x, w, angles, case):
    cos, sin, on = angles
    v, r = x.float(), 1 / torch.sqrt(x.float().square().mean(-1, keepdim=True) + EPS)
    dz = torch.where(on > 0, _rotate(dy.float(), cos, -sin, case), 0.0)
    gr, xhat = dz * w.float(), v * r
    dx = r * (gr - xhat * (gr * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dz * xhat).sum((0, 1))


def _philox_round(words, i):
    c0, c1, c2, c3, k0, k1 = words
    low = 0xFFFFFFFF
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # 64 bits of product, whatever their sign
    return ((b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low,
            k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low)


def _keep_plain(rng, p, m, n):
    """What each value of an [m, n] tensor is multiplied by: 0 or 1 / P(keep)."""
    limit = int(p * 65536 + 0.5)
    count = torch.arange(-(-m * n // 8), device="cuda")
    low = 0xFFFFFFFF
    ones = torch.ones_like(count)
    words = (count & low, count >> 32, ones * (rng[1] & low), ones * (rng[1] >> 32 & low), rng[0] & low, rng[0] >> 32 & low)
    words = torch.stack(functools.reduce(_philox_round, range(7), words)[:4], 1)
    bits = torch.stack((words & 0xFFFF, words >> 16), 2).view(-1)[:m * n].view(m, n)
    return (bits >= limit).float() * (65536 / (65536 - limit))


def _drop_fwd_plain(state):
    case = state["case"]
    x = state["x"]
    h = (state["residual"].float() + x.float() * _keep_plain(state["rng"], case["p"], *x.shape)).to(x.dtype)
    v = h.float()
    if case["norm"] == "rms":
        return h, (v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * state["gamma"].float()).to(x.dtype)
    mean = v.mean(1, keepdim=True)
    v = v - mean
    rstd = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
    return h, (v * rstd * state["gamma"].float() + state["beta"].float()).to(x.dtype), mean[:, 0], rstd[:, 0]


def _norm_bwd_plain(state):
    """The gradient of h in 32 bits, and the parameters'."""
    v, dy = state["h"].float(), state["dy"].float()
    gr = dy * state["gamma"].float()
    if state["case"]["norm"] == "rms":
        rstd = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
        xhat = v * rstd
        d = rstd * (gr - xhat * (gr * xhat).mean(1, keepdim=True))
        return state["dh"].float() + d, (dy * xhat).sum(0)
    rstd = state["rstd"][:, None]
    xhat = (v - state["mean"][:, None]) * rstd
    d = rstd * (gr - gr.mean(1, keepdim=True) - xhat * (gr * xhat).mean(1, keepdim=True))
    return state["dh"].float() + d, (dy * xhat).sum(0), dy.sum(0)


def _run_own(state):
    import row_wise_normalization_ln_gb300 as rn

    case, op = state["case"], state["case"]["op"]
    if op.startswith("rope"):
        q, k = _heads(state["qkv"], case) if case["packed"] else (state["q"], state["k"])
        rest = (q, k, state["wq"], state["wk"], state["cos"], state["sin"], state["pos"], EPS)
        if op == "rope_fwd":
            return rn.rms_fwd_rope(*rest, interleaved=case["interleaved"])
        out_q, out_k = _heads(state["dqkv"], case) if case["packed"] else (None, None)
        return rn.rms_bwd_rope(state["dq"], state["dk"], *rest, interleaved=case["interleaved"], dq_out=out_q, dk_out=out_k)
    p, rng = case["p"], state["rng"]
    if op == "drop_fwd":
        if case["norm"] == "ln":
            return rn.ln_fwd_dropout_add(state["x"], state["residual"], state["gamma"], state["beta"], p, rng, EPS)
        return rn.rms_fwd_dropout_add(state["x"], state["residual"], state["gamma"], p, rng, EPS)
    grads = (state["dy"], state["dh"], state["h"], state["gamma"])
    if op == "drop_bwd":
        if case["norm"] == "ln":
            return rn.ln_bwd_dropout_add(*grads, state["mean"], state["rstd"], p, rng)
        return rn.rms_bwd_dropout_add(*grads, p, rng, EPS)
    if case["norm"] == "ln":
        return rn.ln_bwd_add(*grads, state["mean"], state["rstd"])
    return rn.rms_bwd_add(*grads, EPS)


def run(state):
    if own:
        return _run_own(state)
    case, op = state["case"], state["case"]["op"]
    if op.startswith("rope"):
        q, k = _heads(state["qkv"], case) if case["packed"] else (state["q"], state["k"])
        angles = _angles(state)
        if op == "rope_fwd":
            return _rope_fwd_plain(q, state["wq"], angles, case), _rope_fwd_plain(k, state["wk"], angles, case)
        (dq, dwq), (dk, dwk) = (_rope_bwd_plain(dy, x, w, angles, case) for dy, x, w in
                                ((state["dq"], q, state["wq"]), (state["dk"], k, state["wk"])))
        if case["packed"]:
            out_q, out_k = _heads(state["dqkv"], case)
            dq, dk = out_q.copy_(dq), out_k.copy_(dk)
        return dq, dk, dwq, dwk
    if op == "drop_fwd":
        return _drop_fwd_plain(state)
    d, *columns = _norm_bwd_plain(state)
    if op == "add_bwd":
        return (d.to(state["h"].dtype), *columns)
    dx = d * _keep_plain(state["rng"], case["p"], *d.shape)
    return (dx.to(state["h"].dtype), d.to(state["h"].dtype), *columns)


def work(case):
    e = DTYPES[case["dtype"]].itemsize
    if case["op"].startswith("rope"):
        t, d, heads = case["tokens"], case["width"], case["heads"] + case["kv_heads"]
        table = min(t, case["positions"]) * case["rotary"] * 4 + 8 * t  # the angles of the tokens' positions, and these
        if case["op"] == "rope_fwd":  # q, k, weights in; q, k out
            return {"bytes": 2 * t * heads * d * e + 2 * d * e + table, "flops": t * heads * (4 * d + 3 * case["rotary"])}
        # dq, dk, q, k, weights in; dq, dk, the weights' gradients out
        return {"bytes": 3 * t * heads * d * e + 2 * d * e + 8 * d + table, "flops": t * heads * (12 * d + 3 * case["rotary"])}
    m, n, ln = case["rows"], case["cols"], case["norm"] == "ln"
    stats = 8 * m if ln else 0
    if case["op"] == "drop_fwd":  # x, residual, parameters in; h, y, statistics out
        return {"bytes": 4 * m * n * e + (1 + ln) * n * e + stats + 16, "flops": (10 if ln else 7) * m * n}
    # dy, dh, h, gamma, statistics in; dx, the residual's gradient (one tensor without dropout), column gradients out
    streams = 5 if case["op"] == "drop_bwd" else 4
    return {"bytes": streams * m * n * e + n * e + stats + (1 + ln) * 4 * n + 16, "flops": (14 if ln else 11) * m * n}


def _keep_exact(rng, p, m, n):
    """The mask from the generator's definition, in numpy's unsigned integers."""
    import numpy as np

    limit = math.floor(p * 65536 + 0.5)
    seed, offset = (int(v) for v in rng.tolist())
    c = np.arange(-(-m * n // 8), dtype=np.uint64)
    ctr = [(c % 2**32).astype(np.uint32), (c // 2**32).astype(np.uint32), np.full_like(c, offset % 2**32, dtype=np.uint32),
           np.full_like(c, offset // 2**32, dtype=np.uint32)]
    key = [seed % 2**32, seed // 2**32]
    for _ in range(7):
        a, b = ctr[0].astype(np.uint64) * np.uint64(0xD2511F53), ctr[2].astype(np.uint64) * np.uint64(0xCD9E8D57)
        hi = [(v >> np.uint64(32)).astype(np.uint32) for v in (a, b)]
        ctr = [hi[1] ^ ctr[1] ^ np.uint32(key[0]), b.astype(np.uint32), hi[0] ^ ctr[3] ^ np.uint32(key[1]), a.astype(np.uint32)]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    words = np.empty((c.size, 8), dtype=bool)
    for i, v in enumerate(ctr):
        words[:, 2 * i], words[:, 2 * i + 1] = v % np.uint32(65536) >= limit, v // np.uint32(65536) >= limit
    return torch.from_numpy(words.reshape(-1)[:m * n].reshape(m, n)).cuda(), 65536 / (65536 - limit)


def exact(case, seed):
    state = prepare(case, seed)
    f = torch.float64
    if case["op"].startswith("rope"):
        r, d = case["rotary"], case["width"]
        # a head's rotation as a gather and signs: out[j] = c[j] v[j] + s[j] v[mate[j]], mate and s swapping the pairs
        j = torch.arange(r, device="cuda")
        mate, angle, first = (j ^ 1, j // 2, j % 2 == 0) if case["interleaved"] else ((j + r // 2) % r, j % (r // 2), j < r // 2)
        live = state["pos"] >= 0
        at = state["pos"][live]
        c, s = state["cos"].to(f)[at][:, angle], state["sin"].to(f)[at][:, angle]
        s = torch.where(first, -s, s)[:, None]
        c = c[:, None]
        outs, sums = [], []
        q, k = _heads(state["qkv"], case) if case["packed"] else (state["q"], state["k"])
        for x, w, dy in ((q, "wq", "dq"), (k, "wk", "dk")):
            w, v = state[w].to(f), x[live].to(f)
            r2 = (v * v).sum(-1, keepdim=True) / d + EPS
            out = torch.zeros(x.shape, dtype=f, device="cuda")
            if case["op"] == "rope_fwd":
                v = v * w * r2 ** -0.5
                v[..., :r] = c * v[..., :r] + s * v[..., mate]
                out[live] = v
            else:
                z = state[dy][live].to(f)
                z[..., :r] = c * z[..., :r] - s * z[..., mate]
                sums.append((z * v * r2 ** -0.5).sum((0, 1)))
                z *= w
                out[live] = z * r2 ** -0.5 - v * r2 ** -1.5 * ((z * v).sum(-1, keepdim=True) / d)
            outs.append(out)
        return (*outs, *sums)

    m, n, ln = case["rows"], case["cols"], case["norm"] == "ln"
    gamma, dt = state["gamma"].to(f), DTYPES[case["dtype"]]
    if case["op"] == "drop_fwd":
        keep, scale = _keep_exact(state["rng"], case["p"], m, n)
        h = torch.where(keep, state["x"].to(f) * scale, 0.0) + state["residual"].to(f)
        v = h.to(dt).to(f)  # the norm is that of the sum as it is stored
        if not ln:
            return h, v * gamma * (v.square().mean(1, keepdim=True) + EPS) ** -0.5
        mu = v.sum(1, keepdim=True) / n
        v = v - mu
        rs = (v.square().sum(1, keepdim=True) / n + EPS) ** -0.5
        return h, v * rs * gamma + state["beta"].to(f), mu[:, 0], rs[:, 0]
    dgamma, dbeta = torch.zeros(n, dtype=f, device="cuda"), torch.zeros(n, dtype=f, device="cuda")
    total = []
    # some rows at a time, so that the 64-bit copies stay small
    for a in range(0, m, 8192):
        h, dy, dh = (state[t][a:a + 8192].to(f) for t in ("h", "dy", "dh"))
        if ln:
            rs = state["rstd"][a:a + 8192, None].to(f)
            xh = (h - state["mean"][a:a + 8192, None].to(f)) * rs
        else:
            rs = (h.square().sum(1, keepdim=True) / n + EPS) ** -0.5
            xh = h * rs
        dgamma += (dy * xh).sum(0)
        dbeta += dy.sum(0)
        gr = dy * gamma
        if ln:
            gr -= gr.sum(1, keepdim=True) / n
        total.append(dh + rs * (gr - xh * ((dy * gamma * xh).sum(1, keepdim=True) / n)))
    total = torch.cat(total)
    columns = (dgamma, dbeta) if ln else (dgamma,)
    if case["op"] == "add_bwd":
        return (total, *columns)
    keep, scale = _keep_exact(state["rng"], case["p"], m, n)
    return (torch.where(keep, total * scale, 0.0), total, *columns)
