"""Measured cases of what a decoder block computes between its norms and its
attention: projections with bias, activation and residual, the gated
feed-forward block, and rotary positions of several axes (alone and fused with
the head RMSNorm), forward and backward.

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
def _linear(op, name, T, K, N, dtype="bf16", act="none", bias=False, res=False, save=False, pad=0):
    """op: lin_fwd (res: a residual is added; save: the pre-activation is kept) or lin_bwd."""
    c = {"op": op, "T": T, "K": K, "N": N, "dtype": dtype, "act": act, "bias": bias, "res": res, "save": save, "pad": pad}
    return dict(c, name=name) if name else c


def _gated(op, name, T, K, N, dtype="bf16", act="silu", save=False, pad=0):
    """op: gate_fwd (save: both projections are kept) or gate_bwd; N is the block's inner width."""
    c = {"op": op, "T": T, "K": K, "N": N, "dtype": dtype, "act": act, "save": save, "pad": pad}
    return dict(c, name=name) if name else c


def _axes(op, name, T, Hq, Hk, D, sections, dtype="bf16", interleaved=False, cycled=False, grid=(1, 64, 64), theta=10000.0,
          back=False, zc=False):
    """op: axes (the rotation), axes_norm_fwd or axes_norm_bwd. sections: pairs of each axis, side by side or (cycled)
    dealt in turn; grid: the axes' extents, time outermost."""
    c = {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "sections": ",".join(map(str, sections)), "dtype": dtype,
         "interleaved": interleaved, "cycled": cycled, "grid": ",".join(map(str, grid)), "theta": theta, "back": back, "zc": zc}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a served sequence: the projection behind the attention, added to the residual stream
        _linear("lin_fwd", "linear 1 token", 1, 4096, 4096, res=True),
        # one step of 64 served sequences: q, k and v of 32 + 8 + 8 heads of 128, with a bias
        _linear("lin_fwd", "linear qkv 64 tokens", 64, 4096, 6144, bias=True),
        # a training batch: the first matrix of a plain feed-forward block, its pre-activation kept
        _linear("lin_fwd", "linear 8192 gelu", 8192, 4096, 16384, act="gelu_tanh", bias=True, save=True),
        # the gradients of a square projection of a training batch
        _linear("lin_bwd", "linear bwd 8192", 8192, 4096, 4096),
        # an odd number of rows of odd widths, rows padded apart, all gradients
        _linear("lin_bwd", "linear bwd ragged fp16", 1021, 1000, 2056, dtype="fp16", act="gelu", bias=True, pad=24),
        # one step of 8 served sequences through the gated block: both matrices are read once
        _gated("gate_fwd", "gated 8 tokens", 8, 4096, 14336),
        # the same block over a training batch, both projections kept
        _gated("gate_fwd", "gated 8192", 8192, 4096, 14336, save=True),
        # its gradients
        _gated("gate_bwd", "gated bwd 8192", 8192, 4096, 14336),
        # a small block with odd sizes
        _gated("gate_bwd", "gated bwd ragged fp16", 777, 520, 1384, dtype="fp16", act="gelu_tanh", pad=8),
        # one step of 32 served sequences of text and pictures: head norm, frequencies dealt to time, height, width
        _axes("axes_norm_fwd", "axes norm 32 tokens", 32, 32, 8, 128, (24, 20, 20), cycled=True, grid=(4096, 64, 64),
              theta=5000000.0),
        # a video's latents, 21 frames of 30 x 26: every axis with frequencies of its own, neighbours turned
        _axes("axes", "axes video 16380", 16380, 24, 24, 128, (22, 21, 21), interleaved=True, grid=(21, 30, 26)),
        # a training batch of text and pictures
        _axes("axes_norm_bwd", "axes norm bwd 16384", 16384, 32, 8, 128, (16, 24, 24), grid=(64, 16, 16), theta=1000000.0),
    ]


_MOST_FLOPS = 8 * 8192 * 4096 * 14336  # of the largest listed case
_MOST_BYTES = 2 * (2 * 8192 * 4096 + 4 * 14336 * 4096 + 3 * 8192 * 14336)
_MOST_VALUES = 16384 * 40 * 128        # of one activation of q and k


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("lin_fwd", "lin_bwd", "gate_fwd", "gate_bwd", "axes", "axes_norm_fwd", "axes_norm_bwd"))
    dtype = rng.choice(("bf16", "fp16"))
    if not op.startswith("axes"):
        K = 8 * _log_int(rng, 4, 2048)
        N = 8 * _log_int(rng, 4, min(2048, (1 << 24) // K))  # matrices of 2^27 values and fewer
        per = {"lin_fwd": 2, "lin_bwd": 4, "gate_fwd": 4, "gate_bwd": 8}[op]
        most = min(32768, _MOST_FLOPS // (per * K * N), (_MOST_BYTES - 8 * K * N) // (4 * K + 6 * N))
        T = _log_int(rng, 1, max(1, most))
        pad = rng.choice((0, 0, 8, 64))
        if op.startswith("gate"):
            return _gated(op, None, T, K, N, dtype, rng.choice(("silu", "silu", "gelu_tanh", "gelu", "sigmoid", "relu")),
                          save=op == "gate_fwd" and rng.random() < 0.5, pad=pad)
        act = rng.choice(("none", "none", "gelu", "gelu_tanh", "silu", "relu"))
        return _linear(op, None, T, K, N, dtype, act, bias=rng.random() < 0.5,
                       res=op == "lin_fwd" and rng.random() < 0.5, save=op == "lin_fwd" and act != "none" and rng.random() < 0.5,
                       pad=pad)
    D = rng.choice((64, 80, 96, 128, 128, 192, 256, 8 * rng.randint(4, 64)))
    pairs = D // 2 if rng.random() < 0.6 else rng.randint(4, D // 2)
    n = rng.choice((2, 3, 3))
    first = rng.randint(pairs // (n + 1), pairs - 2 * (n - 1)) if pairs > 8 else pairs - (n - 1)
    rest = pairs - first
    sections = [first] + [rest // (n - 1) + (1 if i < rest % (n - 1) else 0) for i in range(n - 1)]
    cycled = n * max(sections[1:]) <= pairs and rng.random() < 0.5
    Hk = rng.choice((0, 1, 2, 4, 8))
    Hq = rng.choice((1, 4, 8, 16, 24, 5)) if Hk == 0 else Hk * rng.choice((1, 2, 4, 7))
    T = _log_int(rng, 1, max(1, min(65536, _MOST_VALUES // ((Hq + Hk) * D))))
    return _axes(op, None, T, Hq, Hk, D, sections, dtype, interleaved=rng.random() < 0.5, cycled=cycled,
                 grid=[rng.choice((16, 4096, 131072))] + [rng.randint(4, 128) for _ in range(n - 1)],
                 theta=rng.choice((100.0, 10000.0, 5000000.0)), back=op == "axes" and rng.random() < 0.5,
                 zc=op != "axes" and rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _ints(text):
    return [int(v) for v in text.split(",")]


def _axis_of(c):
    """The axis of every pair."""
    sections = _ints(c["sections"])
    n, pairs = len(sections), sum(sections)
    if c["cycled"]:  # time, height, width, time, ... until an axis has its share; the rest is time's
        return [i % n if i < n * sections[i % n] else 0 for i in range(pairs)]
    return [a for a, s in enumerate(sections) for _ in range(s)]


def _inv_freq(c):
    """Neighbours: every axis has frequencies from 1 down, of its own; halves: one ladder over all pairs."""
    sections = _ints(c["sections"])
    if c["interleaved"] and not c["cycled"]:
        f = [c["theta"] ** (-float(i) / s) for s in sections for i in range(s)]
    else:
        f = [c["theta"] ** (-float(i) / sum(sections)) for i in range(sum(sections))]
    return torch.tensor(f, dtype=torch.float64)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[c["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=g)

    def rows(r, n, std=1.0):  # r rows of n values, n + pad apart
        base = torch.zeros((r, n + c["pad"]), dtype=dt, device="cuda")
        if std:
            base[:, :n] = normal(r, n, std=std)
        return base[:, :n]

    s = dict(c)
    T = c["T"]
    if not c["op"].startswith("axes"):
        K, N = c["K"], c["N"]
        s["x"] = rows(T, K)  # a norm's output
        if c["op"].startswith("lin"):
            s["w"] = rows(N, K, std=K ** -0.5)
            if c["op"] == "lin_fwd":
                s["b"] = normal(N, std=0.1) if c["bias"] else None
                s["r"] = rows(T, N, std=2.0) if c["res"] else None
                s["y"] = rows(T, N, std=0)
                s["z"] = rows(T, N, std=0) if c["save"] else None
            else:
                s["g"] = rows(T, N, std=0.1)
                s["z"] = rows(T, N) if c["act"] != "none" else None
                s["dx"], s["dw"] = rows(T, K, std=0), rows(N, K, std=0)
                s["db"] = torch.empty(N, device="cuda") if c["bias"] else None
            return s
        s["wg"], s["wu"] = rows(N, K, std=K ** -0.5), rows(N, K, std=K ** -0.5)
        if c["op"] == "gate_fwd":
            s["h"] = rows(T, N, std=0)
            s["gate"], s["up"] = (rows(T, N, std=0), rows(T, N, std=0)) if c["save"] else (None, None)
        else:
            s["g"], s["gate"], s["up"] = rows(T, N, std=0.1), rows(T, N), rows(T, N)
            s["dx"], s["dwg"], s["dwu"] = rows(T, K, std=0), rows(N, K, std=0), rows(N, K, std=0)
        return s

    D, Hq, Hk = c["D"], c["Hq"], c["Hk"]

    def heads():  # q and k, views of one projection's output
        t = normal(T, (Hq + 2 * Hk) * D).to(dt)
        return t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D) if Hk else None

    s["q"], s["k"] = heads()
    grid = _ints(c["grid"])
    if T <= 256:  # a step of served sequences: a place for each
        at = [torch.randint(0, n, (T,), generator=g, device="cuda") for n in grid]
    else:  # a grid in raster order, from a place of its own on
        i = torch.arange(T, device="cuda") + torch.randint(0, 1000, (1,), generator=g, device="cuda")
        at = []
        for n in reversed(grid[1:]):
            at.insert(0, i % n)
            i = i // n
        at.insert(0, i)
    s["pos"] = torch.stack(at)
    s["inv_freq"] = _inv_freq(c).cuda()
    s["axis"] = torch.tensor(_axis_of(c), dtype=torch.uint8, device="cuda")
    s["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    s["k_out"] = torch.empty((T, Hk, D), dtype=dt, device="cuda") if Hk else None
    if c["op"] == "axes":
        return s
    s["eps"] = 1e-6
    for h, H in (("q", Hq), ("k", Hk)):
        s["w" + h] = normal(D, mean=0.0 if c["zc"] else 1.0, std=0.1) if H else None
        s["rstd_" + h] = torch.empty((T, H), device="cuda") if H else None
        s["dw" + h] = torch.empty(D, device="cuda") if H else None
        if c["op"] == "axes_norm_bwd" and H:
            s["rstd_" + h] = (s[h].double().square().mean(2) + s["eps"]).rsqrt().float()
    if c["op"] == "axes_norm_bwd":
        s["gq"], s["gk"] = heads()
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
_SQRT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def _act(name, z):
    """The activation and its derivative at z, in z's type."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z * (z > 0), (z > 0).to(z.dtype)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    u = z
    if name == "gelu_tanh":  # z sigmoid(2 u): the same function
        u = 2.0 * _SQRT_2_OVER_PI * (z + 0.044715 * z * z * z)
    s, t = 1.0 / (1.0 + torch.exp(-u)), 1.0 / (1.0 + torch.exp(u))  # t = 1 - s
    if name == "sigmoid":
        return s, s * t
    du = 2.0 * _SQRT_2_OVER_PI * (1.0 + 3.0 * 0.044715 * z * z) if name == "gelu_tanh" else 1.0
    return z * s, s + z * s * t * du


def _lin_fwd(s):
    dt = s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(s["act"], z)[0]
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(dt)}
    return dict(out, z=z.to(dt)) if s["save"] else out


def _lin_bwd(s):
    dt = s["x"].dtype
    dz = s["g"].float()
    if s["z"] is not None:
        dz = dz * _act(s["act"], s["z"].float())[1]
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
    return dict(out, db=dz.sum(0)) if s["bias"] else out


def _gate_fwd(s):
    dt, x = s["x"].dtype, s["x"].float()
    gate, up = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    out = {"h": (_act(s["act"], gate)[0] * up).to(dt)}
    return dict(out, gate=gate.to(dt), up=up.to(dt)) if s["save"] else out


def _gate_bwd(s):
    dt, x, g = s["x"].dtype, s["x"].float(), s["g"].float()
    a, da = _act(s["act"], s["gate"].float())
    dgate, dup = g * s["up"].float() * da, g * a
    return {"dx": (dgate @ s["wg"].float() + dup @ s["wu"].float()).to(dt), "dwg": (dgate.t() @ x).to(dt),
            "dwu": (dup.t() @ x).to(dt)}


def _angles(s):
    a = (s["pos"].double()[s["axis"].long()].t() * s["inv_freq"])[:, None]  # far positions: 64 bits
    return a.cos().float(), a.sin().float()


def _rotate(s, x, cos, sin):
    """x's first R values of each head turned by the angles (fp32 in, fp32 out)."""
    R = 2 * s["inv_freq"].shape[0]
    if not s["interleaved"]:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., R:]), -1)


def _turn(s):
    cos, sin = _angles(s)
    if s["back"]:
        sin = -sin
    return {h: _rotate(s, s[h].float(), cos, sin).to(s[h].dtype) for h in ("q", "k") if s[h] is not None}


def _norm_fwd(s):
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


def _norm_bwd(s):
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


_PLAIN = {"lin_fwd": _lin_fwd, "lin_bwd": _lin_bwd, "gate_fwd": _gate_fwd, "gate_bwd": _gate_bwd, "axes": _turn,
          "axes_norm_fwd": _norm_fwd, "axes_norm_bwd": _norm_bwd}


# --------------------------------------------------------------------------
# this package's entry points
# --------------------------------------------------------------------------
def _workspace(s, bytes_of):
    """The backward's scratch, kept by the program between its steps."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(bytes_of(), 16), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    import invariant_rmsnorm_gb300 as rn

    op = s["op"]
    if op == "lin_fwd":
        rn.linear_fwd(s["x"], s["w"], s["b"], s["r"], s["y"], s["z"], s["act"])
        return {"y": s["y"], "z": s["z"]} if s["save"] else {"y": s["y"]}
    if op == "lin_bwd":
        ws = _workspace(s, lambda: rn.linear_bwd_workspace_bytes(s["T"], s["N"], s["K"], s["act"]))
        rn.linear_bwd(s["g"], s["x"], s["w"], s["z"], s["dx"], s["dw"], s["db"], ws, s["act"])
        out = {"dx": s["dx"], "dw": s["dw"]}
        return dict(out, db=s["db"]) if s["bias"] else out
    if op == "gate_fwd":
        rn.linear_gated_fwd(s["x"], s["wg"], s["wu"], s["h"], s["gate"], s["up"], s["act"])
        return {k: s[k] for k in (("h", "gate", "up") if s["save"] else ("h",))}
    if op == "gate_bwd":
        ws = _workspace(s, lambda: rn.linear_gated_bwd_workspace_bytes(s["T"], s["N"], s["K"]))
        rn.linear_gated_bwd(s["g"], s["x"], s["wg"], s["wu"], s["gate"], s["up"], s["dx"], s["dwg"], s["dwu"], ws, s["act"])
        return {k: s[k] for k in ("dx", "dwg", "dwu")}
    have = ("q", "k") if s["k"] is not None else ("q",)
    if op == "axes":
        (rn.rope_axes_bwd if s["back"] else rn.rope_axes_fwd)(s["q"], s["k"], s["inv_freq"], s["axis"], s["q_out"],
                                                              s["k_out"], s["pos"], 1.0, s["interleaved"])
        return {h: s[h + "_out"] for h in have}
    if op == "axes_norm_fwd":
        rn.rmsnorm_rope_axes_fwd(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["axis"], s["q_out"], s["k_out"],
                                 s["rstd_q"], s["rstd_k"], s["pos"], 1.0, s["interleaved"], s["eps"], s["zc"])
        return {**{h: s[h + "_out"] for h in have}, **{"rstd_" + h: s["rstd_" + h] for h in have}}
    ws = _workspace(s, lambda: rn.rmsnorm_rope_bwd_workspace_bytes(s["T"], s["Hq"], s["Hk"], s["D"]))
    rn.rmsnorm_rope_axes_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["axis"], s["rstd_q"],
                             s["rstd_k"], s["q_out"], s["k_out"], s["dwq"], s["dwk"], ws, s["pos"], 1.0, s["interleaved"],
                             s["zc"])
    return {**{"d" + h: s[h + "_out"] for h in have}, **{"dw" + h: s["dw" + h] for h in have}}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    c = case
    T = c["T"]
    if not c["op"].startswith("axes"):
        K, N = c["K"], c["N"]
        if c["op"] == "lin_fwd":
            return {"bytes": 2 * (T * K + N * K + T * N * (1 + c["res"] + c["save"])) + 4 * N * c["bias"], "flops": 2 * T * N * K}
        if c["op"] == "lin_bwd":
            return {"bytes": 2 * (2 * T * K + 2 * N * K + T * N * (1 + (c["act"] != "none"))) + 4 * N * c["bias"],
                    "flops": 4 * T * N * K}
        if c["op"] == "gate_fwd":
            return {"bytes": 2 * (T * K + 2 * N * K + T * N * (1 + 2 * c["save"])), "flops": 4 * T * N * K}
        return {"bytes": 2 * (2 * T * K + 4 * N * K + 3 * T * N), "flops": 8 * T * N * K}
    H, D, sections = c["Hq"] + c["Hk"], c["D"], _ints(c["sections"])
    n, pairs, tensors = T * H * D, sum(sections), 2 if c["Hk"] else 1
    angles = 8 * T * len(sections) + 9 * pairs
    turn = 6 * T * H * pairs + 4 * T * pairs
    if c["op"] == "axes":
        return {"bytes": 4 * n + angles, "flops": turn}
    rows = 4 * T * H
    if c["op"] == "axes_norm_fwd":
        return {"bytes": 4 * n + angles + rows + 4 * tensors * D, "flops": turn + 4 * n}
    return {"bytes": 6 * n + angles + rows + 8 * tensors * D, "flops": turn + 10 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
_TORCH_ACT = {
    "none": lambda z: z.clone(),
    "relu": torch.relu,
    "silu": lambda z: z / (1.0 + torch.exp(-z)),
    "sigmoid": torch.sigmoid,
    "gelu": lambda z: z * torch.special.ndtr(z),
    "gelu_tanh": lambda z: 0.5 * z * (1.0 + torch.tanh(_SQRT_2_OVER_PI * z * (1.0 + 0.044715 * z.pow(2)))),
}


def _with_slope(act, z):
    """The activation of z and its slope there, by automatic differentiation."""
    z = z.clone().requires_grad_()
    a = _TORCH_ACT[act](z)
    slope, = torch.autograd.grad(a.sum(), z)
    return a.detach(), slope


def exact(case, seed):
    s = prepare(case, seed)
    up = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = s["op"]
    if op == "lin_fwd":
        z = torch.einsum("tk,nk->tn", up["x"], up["w"])
        if s["b"] is not None:
            z = z + up["b"]
        y = _TORCH_ACT[s["act"]](z)
        if s["r"] is not None:
            y = y.add_(up["r"])
        return {"y": y, "z": z} if s["save"] else {"y": y}
    if op == "lin_bwd":
        dz = up["g"] if s["z"] is None else up["g"] * _with_slope(s["act"], up["z"])[1]
        out = {"dx": torch.einsum("tn,nk->tk", dz, up["w"]), "dw": torch.einsum("tn,tk->nk", dz, up["x"])}
        return dict(out, db=torch.einsum("tn->n", dz)) if s["bias"] else out
    if op == "gate_fwd":
        gate = torch.einsum("tk,nk->tn", up["x"], up["wg"])
        upper = torch.einsum("tk,nk->tn", up["x"], up["wu"])
        out = {"h": _TORCH_ACT[s["act"]](gate).mul_(upper)}
        return dict(out, gate=gate, up=upper) if s["save"] else out
    if op == "gate_bwd":
        a, slope = _with_slope(s["act"], up["gate"])
        dup, dgate = a.mul_(up["g"]), slope.mul_(up["g"]).mul_(up["up"])
        return {"dx": torch.einsum("tn,nk->tk", dgate, up["wg"]).add_(torch.einsum("tn,nk->tk", dup, up["wu"])),
                "dwg": torch.einsum("tn,tk->nk", dgate, up["x"]), "dwu": torch.einsum("tn,tk->nk", dup, up["x"])}
    # a pair (a, b) is the number a + i b, turned by exp(i * angle)
    D, n = s["D"], s["inv_freq"].shape[0]
    angle = torch.stack([up["pos"][a].double() * f for a, f in zip(s["axis"].tolist(), up["inv_freq"])], 1)
    turn = torch.polar(torch.ones_like(angle), angle)
    if s["back"] or op == "axes_norm_bwd":
        turn = turn.conj()
    i = torch.arange(n, device="cuda")
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + n)

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
        if op == "axes":
            out[h] = turned(x)
            continue
        w = (s["w" + h] + 1.0).double() if s["zc"] else up["w" + h]  # the +1 is one of 32 bits
        if op == "axes_norm_fwd":
            r = torch.pow((x * x).sum(2) / D + float(torch.tensor(s["eps"], dtype=torch.float32)), -0.5)
            out[h] = turned(x * w * r.unsqueeze(2))
            out["rstd_" + h] = r
            continue
        g, r = turned(up["g" + h]), up["rstd_" + h].unsqueeze(2)
        out["dw" + h] = torch.einsum("thd,thd->d", g, x * r)
        dot = torch.einsum("thd,thd,d->th", g, x, w).unsqueeze(2)
        out["d" + h] = g * w * r - x * dot * r.pow(3) / D
    return out
