"""Measured cases of the operators around a decoder block's projections and
attention: LayerNorm forward and backward, rotary positions on q and k, and the
head RMSNorm of q and k fused with their rotary positions, forward and backward.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, angles in 64) or, with ``own`` set, through this package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _ln(op, name, T, D, dtype="bf16", bias=True, zc=False, pad=0, shift=0.0):
    c = {"op": op, "T": T, "D": D, "dtype": dtype, "bias": bias, "zc": zc, "pad": pad, "shift": shift}
    return dict(c, name=name) if name else c


def _heads(op, name, T, Hq, Hk, D, R, dtype="bf16", layout="half", span=4096, theta=10000.0, factor=1.0, back=False,
           zc=False, fused_qkv=True):
    c = {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "dtype": dtype, "layout": layout, "span": span,
         "theta": theta, "factor": factor, "back": back, "zc": zc, "fused_qkv": fused_qkv}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a served sequence: a norm before each projection, where latency counts
        _ln("ln_fwd", "ln fwd 1 token", 1, 4096),
        # this repository's benchmark shape: a training or prompt batch at a common width
        _ln("ln_fwd", "ln fwd 32768x4096", 32768, 4096),
        # a norm over each head's values: very many short rows, no bias
        _ln("ln_fwd", "ln fwd heads fp16", 262144, 128, dtype="fp16", bias=False),
        # the training step of the benchmark shape, weight and bias gradients
        _ln("ln_bwd", "ln bwd 32768x4096", 32768, 4096),
        # an odd number of rows of an odd width, rows padded apart, a mean far from zero
        _ln("ln_bwd", "ln bwd ragged fp16", 4099, 5000, dtype="fp16", zc=True, pad=24, shift=3.0),
        # the gradient of the head norm
        _ln("ln_bwd", "ln bwd heads", 262144, 128, bias=False),
        # one step of 16 served sequences, positions far into a scaled context
        _heads("rope", "rope 16 tokens", 16, 32, 8, 128, 128, span=1000000, theta=500000.0, factor=8.0),
        # the gradient of a training batch: interleaved pairs in part of the head
        _heads("rope", "rope bwd interleaved", 16381, 32, 32, 80, 32, dtype="fp16", layout="interleaved", span=8192,
               back=True),
        # one step of 64 served sequences: wide heads, few of k, a quarter rotated
        _heads("rr_fwd", "norm+rope 64 tokens", 64, 16, 2, 256, 64, span=262144, theta=10000000.0, zc=True),
        # a prompt or training batch, whole heads rotated
        _heads("rr_fwd", "norm+rope 16384", 16384, 32, 8, 128, 128, span=16384, theta=1000000.0),
        # the training steps of both head shapes
        _heads("rr_bwd", "norm+rope bwd 16384", 16384, 32, 8, 128, 128, span=16384, theta=1000000.0),
        _heads("rr_bwd", "norm+rope bwd 256", 4093, 16, 2, 256, 64, dtype="fp16", span=4096, theta=10000000.0, zc=True),
    ]


_MOST = 32768 * 4096  # values of one activation in the largest listed case


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "rope", "rr_fwd", "rr_bwd"))
    dtype = rng.choice(("bf16", "fp16"))
    if op.startswith("ln"):
        D = 8 * _log_int(rng, 4, 2048)
        T = _log_int(rng, 1, max(1, min(1 << 19, _MOST // D)))
        return _ln(op, None, T, D, dtype, bias=rng.random() < 0.7, zc=rng.random() < 0.3,
                   pad=rng.choice((0, 0, 8, 64)), shift=rng.choice((0.0, 1.0, 5.0)))
    D = rng.choice((64, 64, 80, 96, 128, 128, 128, 192, 256, 8 * rng.randint(4, 64)))
    layout = rng.choice(("half", "interleaved"))
    R = D if rng.random() < 0.5 else 2 * rng.randint(4, D // 2)
    Hk = rng.choice((0, 1, 2, 4, 8))
    Hq = rng.choice((1, 4, 8, 16, 32, 5)) if Hk == 0 else Hk * rng.choice((1, 2, 4, 7))
    T = _log_int(rng, 1, max(1, min(65536, _MOST // 2 // ((Hq + Hk) * D))))
    return _heads(op, None, T, Hq, Hk, D, R, dtype, layout, span=_log_int(rng, max(T, 16), 1 << 20),
                  theta=rng.choice((10000.0, 500000.0, 10000000.0)), factor=rng.choice((1.0, 1.0, 4.0, 16.0)),
                  back=op == "rope" and rng.random() < 0.5, zc=op != "rope" and rng.random() < 0.5,
                  fused_qkv=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _inv_freq(c):
    """The frequencies of the R/2 pairs; with a factor, slow pairs (fewer than
    4 turns over the original length) are interpolated, fast ones (more than 32)
    kept, and the attention's scale grows with the factor."""
    n = c["R"] // 2
    f = [c["theta"] ** (-2.0 * i / c["R"]) for i in range(n)]
    if c["factor"] > 1.0:
        length = 8192.0
        keep = [min(1.0, max(0.0, (length * v / (2.0 * math.pi) - 4.0) / (32.0 - 4.0))) for v in f]
        f = [v * (k + (1.0 - k) / c["factor"]) for v, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64)


def _scale(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["factor"] > 1.0 else 1.0


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[c["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=g)

    def new(*shape):
        return torch.empty(shape, device="cuda")

    s = dict(c)
    if c["op"].startswith("ln"):
        T, D = c["T"], c["D"]

        def rows(t):  # rows D + pad apart
            base = torch.zeros((T, D + c["pad"]), dtype=dt, device="cuda")
            base[:, :D] = t
            return base[:, :D]

        s["x"] = rows(normal(T, D, mean=c["shift"]) * (1.0 + 0.5 * normal(T, 1).abs()))
        s["w"] = normal(D, mean=0.0 if c["zc"] else 1.0, std=0.1)
        s["b"] = normal(D, std=0.1) if c["bias"] else None
        s["eps"] = 1e-5
        s["out"] = rows(torch.zeros((), device="cuda"))
        if c["op"] == "ln_fwd":
            s["mean"], s["rstd"] = new(T), new(T)
        else:
            xd = s["x"].double()
            mean = xd.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((xd - mean[:, None]).square_().mean(1) + s["eps"]).rsqrt().float()
            s["g"] = rows(normal(T, D))
            s["dw"] = new(D)
            s["db"] = new(D) if c["bias"] else None
        return s

    T, D, Hq, Hk = c["T"], c["D"], c["Hq"], c["Hk"]

    def heads():  # q and k, views of one projection's output or tensors of their own
        if c["fused_qkv"]:
            t = normal(T, (Hq + 2 * Hk) * D).to(dt)
            return t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D) if Hk else None
        return normal(T, Hq, D).to(dt), normal(T, Hk, D).to(dt) if Hk else None

    s["q"], s["k"] = heads()
    if T <= 256:  # a step of served sequences: a position for each
        s["pos"] = torch.randint(0, c["span"], (T,), generator=g, device="cuda")
    else:  # packed sequences, each counted from its own start
        cut = torch.randint(1, T, (3,), generator=g, device="cuda").sort().values
        at = torch.arange(T, device="cuda")
        start = torch.zeros(T, dtype=torch.int64, device="cuda")
        for i in range(3):
            start = torch.where(at >= cut[i], cut[i], start)
        s["pos"] = (at - start) % c["span"]
    s["inv_freq"] = _inv_freq(c).cuda()
    s["scale"] = _scale(c)
    s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    s["k_out"] = torch.empty((T, Hk, D), dtype=dt, device="cuda") if Hk else None
    if c["op"] == "rope":
        return s
    s["eps"] = 1e-6
    for h, H in (("q", Hq), ("k", Hk)):
        s["w" + h] = normal(D, mean=0.0 if c["zc"] else 1.0, std=0.1) if H else None
        s["rstd_" + h] = new(T, H) if H else None
        if c["op"] == "rr_bwd" and H:
            s["rstd_" + h] = (s[h].double().square().mean(2) + s["eps"]).rsqrt().float()
        s["dw" + h] = new(D) if H else None
    if c["op"] == "rr_bwd":
        s["gq"], s["gk"] = heads()
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(xc.square().mean(1) + s["eps"])
    y = xc * rstd[:, None] * (s["w"] + 1.0 if s["zc"] else s["w"])
    if s["b"] is not None:
        y = y + s["b"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _ln_bwd(s):
    g, rstd = s["g"].float(), s["rstd"][:, None]
    n = (s["x"].float() - s["mean"][:, None]) * rstd
    gw = g * (s["w"] + 1.0 if s["zc"] else s["w"])
    dx = rstd * (gw - gw.mean(1, keepdim=True) - n * (gw * n).mean(1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype), "dw": (g * n).sum(0)}
    if s["b"] is not None:
        out["db"] = g.sum(0)
    return out


def _angles(s):
    a = s["pos"].double()[:, None, None] * s["inv_freq"]  # far positions: 64 bits
    return (a.cos() * s["scale"]).float(), (a.sin() * s["scale"]).float()


def _rotate(s, x, cos, sin):
    """x's first R values of each head turned by the angles (fp32 in, fp32 out)."""
    R = s["R"]
    if s["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., R:]), -1)


def _rope(s):
    cos, sin = _angles(s)
    if s["back"]:
        sin = -sin
    return {h: _rotate(s, s[h].float(), cos, sin).to(s[h].dtype) for h in ("q", "k") if s[h] is not None}


def _rr_fwd(s):
    cos, sin = _angles(s)
    out = {}
    for h in ("q", "k"):
        if s[h] is not None:
            x = s[h].float()
            rstd = 1.0 / torch.sqrt(x.square().mean(2) + s["eps"])
            w = s["w" + h] + 1.0 if s["zc"] else s["w" + h]
            out[h] = _rotate(s, x * rstd[..., None] * w, cos, sin).to(s[h].dtype)
            out["rstd_" + h] = rstd
    return out


def _rr_bwd(s):
    cos, sin = _angles(s)
    out = {}
    for h in ("q", "k"):
        if s[h] is not None:
            g = _rotate(s, s["g" + h].float(), cos, -sin)
            rstd = s["rstd_" + h][..., None]
            n = s[h].float() * rstd
            gw = g * (s["w" + h] + 1.0 if s["zc"] else s["w" + h])
            dx = rstd * (gw - n * (gw * n).mean(2, keepdim=True))
            out["d" + h] = dx.to(s[h].dtype)
            out["dw" + h] = (g * n).sum((0, 1))
    return out


_PLAIN = {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "rope": _rope, "rr_fwd": _rr_fwd, "rr_bwd": _rr_bwd}


# --------------------------------------------------------------------------
# this package's entry points
# --------------------------------------------------------------------------
def _workspace(s, bytes_of):
    """The weight gradients' scratch, kept by the program between its steps."""
    if "ws" not in s:
        s["ws"] = torch.empty(bytes_of(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    import invariant_rmsnorm_gb300 as rn

    op = s["op"]
    if op == "ln_fwd":
        rn.layernorm_fwd(s["x"], s["w"], s["b"], s["out"], s["mean"], s["rstd"], s["eps"], s["zc"])
        return {"y": s["out"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_bwd":
        ws = _workspace(s, lambda: rn.layernorm_bwd_workspace_bytes(s["T"], s["D"]))
        rn.layernorm_bwd(s["g"], s["x"], s["w"], s["mean"], s["rstd"], s["out"], s["dw"], s["db"], ws, s["zc"])
        out = {"dx": s["out"], "dw": s["dw"]}
        return out if s["db"] is None else dict(out, db=s["db"])
    inter = s["layout"] == "interleaved"
    have = ("q", "k") if s["k"] is not None else ("q",)
    if op == "rope":
        (rn.rope_bwd if s["back"] else rn.rope_fwd)(s["q"], s["k"], s["inv_freq"], s["q_out"], s["k_out"], s["pos"],
                                                    s["scale"], inter)
        return {h: s[h + "_out"] for h in have}
    if op == "rr_fwd":
        rn.rmsnorm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["q_out"], s["k_out"], s["rstd_q"],
                            s["rstd_k"], s["pos"], s["scale"], inter, s["eps"], s["zc"])
        return {**{h: s[h + "_out"] for h in have}, **{"rstd_" + h: s["rstd_" + h] for h in have}}
    ws = _workspace(s, lambda: rn.rmsnorm_rope_bwd_workspace_bytes(s["T"], s["Hq"], s["Hk"], s["D"]))
    rn.rmsnorm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["rstd_q"], s["rstd_k"],
                        s["q_out"], s["k_out"], s["dwq"], s["dwk"], ws, s["pos"], s["scale"], inter, s["zc"])
    return {**{"d" + h: s[h + "_out"] for h in have}, **{"dw" + h: s["dw" + h] for h in have}}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"].startswith("ln"):
        n, vec = c["T"] * c["D"], 4 * c["D"] * (2 if c["bias"] else 1)
        if c["op"] == "ln_fwd":
            return {"bytes": 4 * n + 8 * c["T"] + vec, "flops": 8 * n}
        return {"bytes": 6 * n + 8 * c["T"] + 4 * c["D"] + vec, "flops": 14 * n}
    H = c["Hq"] + c["Hk"]
    n, tensors = c["T"] * H * c["D"], 2 if c["Hk"] else 1
    angles = 8 * c["T"] + 4 * c["R"]
    turn = 3 * c["T"] * H * c["R"] + 2 * c["T"] * c["R"]
    if c["op"] == "rope":
        return {"bytes": 4 * n + angles, "flops": turn}
    rows = 4 * c["T"] * H
    if c["op"] == "rr_fwd":
        return {"bytes": 4 * n + angles + rows + 4 * tensors * c["D"], "flops": turn + 4 * n}
    return {"bytes": 6 * n + angles + rows + 8 * tensors * c["D"], "flops": turn + 10 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    up = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if s["op"].startswith("ln"):
        x, w, D = up["x"], up["w"], s["D"]
        w = (s["w"] + 1.0).double() if s["zc"] else w  # the +1 is one of 32 bits
        if s["op"] == "ln_fwd":
            m = x.sum(1) / D
            x = x - m.unsqueeze(1)
            r = torch.pow((x * x).sum(1) / D + float(torch.tensor(s["eps"], dtype=torch.float32)), -0.5)
            y = x.mul_(r.unsqueeze(1)).mul_(w)
            return {"y": y if s["b"] is None else y.add_(up["b"]), "mean": m, "rstd": r}
        g, r = up["g"], up["rstd"].unsqueeze(1)
        n = (x - up["mean"].unsqueeze(1)) * r
        out = {"dw": torch.einsum("td,td->d", g, n)}
        if s["b"] is not None:
            out["db"] = torch.einsum("td->d", g)
        a = (g @ w).unsqueeze(1) / D  # mean of g w
        b = torch.einsum("td,td,d->t", g, n, w).unsqueeze(1) / D  # mean of g w n
        out["dx"] = (g * w).sub_(a).sub_(n.mul_(b)).mul_(r)
        return out
    # a pair (a, b) is the number a + i b, turned by scale * exp(i * angle)
    R, D, T = s["R"], s["D"], s["T"]
    angle = s["pos"].double().unsqueeze(1) * up["inv_freq"].unsqueeze(0)
    turn = torch.polar(torch.full_like(angle, float(torch.tensor(s["scale"], dtype=torch.float32))), angle)
    if s["back"] or s["op"] == "rr_bwd":
        turn = turn.conj()
    i = torch.arange(R // 2, device="cuda")
    first, second = (i, i + R // 2) if s["layout"] == "half" else (2 * i, 2 * i + 1)

    def turned(t):
        t = t.clone()
        z = torch.complex(t[:, :, first], t[:, :, second]) * turn.unsqueeze(1)
        t[:, :, first], t[:, :, second] = z.real, z.imag
        return t

    out = {}
    for h in ("q", "k"):
        if s[h] is None:
            continue
        x = up[h]
        if s["op"] == "rope":
            out[h] = turned(x)
            continue
        w = (s["w" + h] + 1.0).double() if s["zc"] else up["w" + h]
        if s["op"] == "rr_fwd":
            r = torch.pow((x * x).sum(2) / D + float(torch.tensor(s["eps"], dtype=torch.float32)), -0.5)
            out[h] = turned(x * w * r.unsqueeze(2))
            out["rstd_" + h] = r
            continue
        g, r = turned(up["g" + h]), up["rstd_" + h].unsqueeze(2)
        out["dw" + h] = torch.einsum("thd,thd->d", g, x * r)
        dot = torch.einsum("thd,thd,d->th", g, x, w).unsqueeze(2)
        out["d" + h] = g * w * r - x * dot * r.pow(3) / D
    return out
