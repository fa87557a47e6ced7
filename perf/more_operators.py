"""Measured cases of the operators between a transformer layer's quantized
products: the gated feed-forward product with its gradient, the norms before and
after a block joined with its gate and residual scale, and rotary positions.

A case is a dict of plain values; `prepare` makes its tensors on the GPU from a
seed, `run` makes one pass: in plain torch operations in 32 bits (angles in 64), or,
with `own` set, through learnable_scale_fake_gb300.aqfq.  `exact` restates each
operator in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # one token through one expert's gate and up projections: latency
        dict(name="gated_token", kind="gated_fwd", M=1, N=768, K=2048, act="silu"),
        # a prompt through the feed-forward block of a 2048-wide model
        dict(name="gated_prompt", kind="gated_fwd", M=4096, N=8192, K=2048, act="silu"),
        # a ragged batch, sizes that no tile divides
        dict(name="gated_ragged", kind="gated_fwd", M=1000, N=1544, K=776, act="gelu_tanh"),
        # a training step of the whole block up to its down projection: forward with gate and up
        # kept in 8 bits, the gradient through the down projection and the gate, the input's and
        # both weights' gradients
        dict(name="gated_train", kind="gated_train", M=4096, N=8192, K=2048, D=2048, act="silu",
             fmt="int8", group=128),
        # a small ragged step whose hidden activation is fake-quantized before the down
        # projection, so that its gradient arrives as a tensor of its own
        dict(name="gated_act_train", kind="gated_act_train", M=515, N=776, K=1032, act="gelu",
             fmt="e4m3", group=64),
        # one token between two blocks of a 2048-wide model: pure latency
        dict(name="join_token", kind="join_fwd", rows=1, cols=2048, dtype="bf16", post=True,
             gate=True),
        # a prompt between two blocks: norm after, gate, residual, norm before, in one pass
        dict(name="join_prompt", kind="join_fwd", rows=8192, cols=4096, dtype="bf16", post=True,
             gate=True),
        # a training step of the same join
        dict(name="join_train", kind="join_train", rows=8192, cols=4096, dtype="bf16", post=True,
             gate=True),
        # odd sizes in 32 bits without the norm after the block: rows that no wide load fits
        dict(name="join_train_odd", kind="join_train", rows=1537, cols=1003, dtype="f32", post=False,
             gate=True),
        # queries and keys of one token far into a long context
        dict(name="rotary_token", kind="rotary", T=1, Hq=32, Hk=8, D=128, rot=128, layout="half",
             scaling="parts", dtype="bf16", transposed=False, far=True),
        # queries and keys of 65536 tokens, sequences one after another
        dict(name="rotary_prompt", kind="rotary", T=65536, Hq=32, Hk=8, D=128, rot=128,
             layout="half", scaling="none", dtype="bf16", transposed=False, far=False),
        # gradient through interleaved pairs on a part of each head, sizes that no wide load fits
        dict(name="rotary_odd", kind="rotary", T=1537, Hq=12, Hk=3, D=80, rot=42,
             layout="interleaved", scaling="linear", dtype="f32", transposed=True, far=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log8(rng, lo, hi):
    return 8 * _log(rng, lo // 8, hi // 8)


def draw(rng):
    kind = rng.choice(["gated_fwd", "gated_fwd", "gated_train", "gated_act_train", "gated_dgrad",
                       "join_fwd", "join_train", "join_train", "rotary", "rotary"])
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu", "silu"])
    fmt = rng.choice(["int8", "e4m3"])
    group = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind.startswith("gated"):
        while True:
            few = kind == "gated_fwd" and rng.random() < 0.4
            M = _log(rng, 1, 64) if few else _log(rng, 64, 8192)
            N, K, D = (_log8(rng, 256, 8192) for _ in range(3))
            if M * N * max(K, D) <= 4096 * 8192 * 2048:
                break
        c = dict(kind=kind, M=M, N=N, K=K, act=act)
        if kind == "gated_fwd":
            return c
        if kind in ("gated_train", "gated_dgrad"):
            c["D"] = D
        return dict(c, fmt=fmt, group=group)
    if kind.startswith("join"):
        rows = _log(rng, 1 if kind == "join_fwd" else 16, 16384)
        cols = _log(rng, 64, 8192) if rng.random() < 0.4 else _log8(rng, 64, 8192)
        return dict(kind=kind, rows=rows, cols=cols, dtype=dtype, post=rng.random() < 0.7,
                    gate=rng.random() < 0.7)
    D = rng.choice([64, 80, 96, 128, 192, 256])
    Hk = rng.choice([1, 2, 3, 4, 8])
    return dict(kind=kind, T=_log(rng, 1, 65536 * 2048 // (D * Hk * 16)), Hq=Hk * rng.choice([1, 3, 4, 8]),
                Hk=Hk, D=D, rot=rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]),
                layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "ntk", "parts"]), dtype=dtype,
                transposed=rng.random() < 0.4, far=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------------

def _normal(g, shape, std, dtype=torch.bfloat16, outliers=0.0):
    t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std
    if outliers:  # a share of values 30 times as large, as activations have them
        t = torch.where(torch.rand(shape, generator=g, device="cuda") < outliers, t * 30.0, t)
    return t.to(dtype)


def _frequencies(rot, scaling, base=10000.0, factor=4.0, length=8192.0, low=1.0, high=32.0):
    """Angle per position of each pair, in 64 bits, and the factor on cosine and sine."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        keep = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f, 0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c, s = case, {"case": dict(case)}
    kind = c["kind"]

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if kind.startswith("join"):
        R, C = c["rows"], c["cols"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # a residual stream with outliers, and the block's output
        s["x"], s["f"] = _normal(g, (R, C), 2.0, dt, 1e-3), _normal(g, (R, C), 0.7, dt)
        s["gamma_post"] = (1.0 + _normal(g, (C,), 0.1, torch.float32)).to(dt) if c["post"] else None
        s["gate"] = _normal(g, (C,), 0.5, dt) if c["gate"] else None
        s["gamma_pre"] = (1.0 + _normal(g, (C,), 0.1, torch.float32)).to(dt)
        s["alpha"] = 0.5
        s["h"], s["y"] = empty(R, C, dtype=dt), empty(R, C, dtype=dt)
        s["rstd_pre"] = empty(R, dtype=torch.float32)
        s["rstd_post"] = empty(R, dtype=torch.float32) if c["post"] else None
        if kind == "join_train":
            s["dy"], s["dh"] = _normal(g, (R, C), 1.0, dt), _normal(g, (R, C), 1.0, dt)
            s["dx"], s["df"] = empty(R, C, dtype=dt), empty(R, C, dtype=dt)
            s["dgamma_pre"] = empty(C, dtype=torch.float32)
            s["dgamma_post"] = empty(C, dtype=torch.float32) if c["post"] else None
            s["dgate"] = empty(C, dtype=torch.float32) if c["gate"] else None
            s["workspace"] = empty(32 << 20, dtype=torch.uint8)
        return s
    if kind == "rotary":
        T, D = c["T"], c["D"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        for name, H in (("q", c["Hq"]), ("k", c["Hk"])):
            std = torch.exp(torch.rand((H, 1), generator=g, device="cuda") * math.log(100.0)) * 0.1
            s[name] = (torch.randn((T, H, D), generator=g, device="cuda") * std).to(dt)
            s["y" + name] = empty(T, H, D, dtype=dt)
        # sequences one after another, or single tokens far into their contexts
        if c["far"]:
            s["pos"] = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda")
        else:
            s["pos"] = torch.arange(T, device="cuda") % max(1, (T * 3 + 3) // 4)
        f, s["mscale"] = _frequencies(c["rot"], c["scaling"])
        s["freqs"] = f.cuda()
        return s
    M, N, K = c["M"], c["N"], c["K"]
    s["y"] = empty(M, N)
    s["workspace"] = empty(96 << 20, dtype=torch.uint8)  # for the largest need of the case's calls
    if kind != "gated_dgrad":
        s["x"] = _normal(g, (M, K), 1.0)
        s["w"] = _normal(g, (2 * N, K), K ** -0.5)  # gate rows, then up rows
    if kind in ("gated_train", "gated_dgrad"):
        s["dz"], s["w2"] = _normal(g, (M, c["D"]), 1.0), _normal(g, (c["D"], N), N ** -0.5)
    if kind == "gated_act_train":
        s["dy"] = _normal(g, (M, N), 1.0)
    if kind != "gated_fwd":
        s["dp"], s["hidden"] = empty(M, 2 * N), empty(M, N)
        n = -(-N // c["group"])
        for name in ("gate", "up"):
            if kind == "gated_dgrad":  # kept by an earlier forward
                q, scale = _quantize(_normal(g, (M, N), 1.0, torch.float32, 1e-3), c["fmt"], c["group"])
                q = q[:, :N].contiguous()
                q = q.to(torch.int8) if c["fmt"] == "int8" else q.to(torch.float8_e4m3fn)
                s[name] = (q.view(torch.uint8), scale)
            else:
                s[name] = (empty(M, N, dtype=torch.uint8), empty(M, n, dtype=torch.float32))
        if kind != "gated_dgrad":
            s["dx"], s["dw"] = empty(M, K), empty(2 * N, K)
        if kind == "gated_train":
            s["dw2"] = empty(c["D"], N)
    return s


# ---- plain forms ---------------------------------------------------------------------

def _act(p, act):
    if act == "relu":
        return torch.clamp(p, min=0.0)
    if act == "gelu":
        return 0.5 * p * (1.0 + torch.erf(p * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * p * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (p + 0.044715 * p * p * p)))
    return p / (1.0 + torch.exp(-p))


def _dact(p, act):
    if act == "relu":
        return (p > 0).to(p.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(p * math.sqrt(0.5)))
                + p * torch.exp(-0.5 * p * p) * (1.0 / math.sqrt(2.0 * math.pi)))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (p + 0.044715 * p * p * p))
        return 0.5 * (1.0 + t) + 0.5 * p * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * p * p)
    sg = 1.0 / (1.0 + torch.exp(-p))
    return sg * (1.0 + p * (1.0 - sg))


def _quantize(x, fmt, group):
    """Grid values [rows, cols padded to the group] and scales of x (float32)."""
    R, C = x.shape
    n = -(-C // group)
    p = torch.zeros((R, n * group), dtype=torch.float32, device=x.device)
    p[:, :C] = x
    p = p.view(R, n, group)
    amax = p.abs().amax(2)
    scale = amax / torch.full_like(amax, QMAX[fmt])
    v = torch.where(scale[:, :, None] > 0, p / scale[:, :, None], torch.zeros_like(p))
    v = v.clamp(-QMAX[fmt], QMAX[fmt])
    q = torch.round(v) if fmt == "int8" else v.to(torch.float8_e4m3fn).to(torch.float32)
    return q.view(R, n * group), scale


def _dequantize(q, scale, C, group):
    return (q.view(q.shape[0], -1, group) * scale[:, :, None]).view(q.shape[0], -1)[:, :C]


def _stored(kept, fmt, group):
    q = kept[0].view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).to(torch.float32)
    C = q.shape[1]
    pad = kept[1].shape[1] * group - C
    if pad:
        q = torch.cat([q, torch.zeros((q.shape[0], pad), device=q.device)], 1)
    return _dequantize(q, kept[1], C, group)


def _plain_join(s):
    c = s["case"]
    dt = s["x"].dtype
    one = torch.ones((), device=s["x"].device)
    f, x, gpre = s["f"].float(), s["x"].float(), s["gamma_pre"].float()
    gate = s["gate"].float() if c["gate"] else one
    out = {}
    if c["post"]:
        gpost = s["gamma_post"].float()
        out["rstd_post"] = r = torch.rsqrt((f * f).mean(1) + EPS)
        n = f * r[:, None]
    else:
        gpost, n = one, f
    h = x + s["alpha"] * (gate * (n * gpost))
    r = torch.rsqrt((h * h).mean(1) + EPS)
    out.update(h=h.to(dt), y=(h * r[:, None] * gpre).to(dt), rstd_pre=r)
    if c["kind"] == "join_fwd":
        return out
    dy, hh = s["dy"].float(), h.to(dt).float() * r[:, None]  # h is kept in its own type
    u = dy * gpre
    dx = r[:, None] * (u - hh * (u * hh).mean(1)[:, None]) + s["dh"].float()
    out["dgamma_pre"] = (dy * hh).sum(0)
    share = (dx * n).sum(0)
    if c["gate"]:
        out["dgate"] = s["alpha"] * gpost * share
    v = s["alpha"] * (dx * (gate * gpost))
    if c["post"]:
        out["dgamma_post"] = s["alpha"] * gate * share
        v = out["rstd_post"][:, None] * (v - n * (v * n).mean(1)[:, None])
    out.update(dx=dx.to(dt), df=v.to(dt))
    return out


def _plain_rotary(s):
    c, out = s["case"], {}
    a = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = torch.cos(a) * s["mscale"], torch.sin(a) * s["mscale"]
    cos, sin = cos.float()[:, None], (-sin if c["transposed"] else sin).float()[:, None]
    half = c["rot"] // 2
    for name in ("q", "k"):
        x = s[name].float()
        y = x.clone()
        if c["layout"] == "half":
            lo, hi = slice(0, half), slice(half, 2 * half)
        else:
            lo, hi = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
        p, q = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = p * cos - q * sin, p * sin + q * cos
        out[name] = y.to(s[name].dtype)
    return out


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind.startswith("join"):
        return _plain_join(s)
    if kind == "rotary":
        return _plain_rotary(s)
    out = {}
    if kind != "gated_dgrad":
        N = c["N"]
        x, w = s["x"].float(), s["w"].float()
        p = torch.matmul(x, w.t())
        g, u = p[:, :N], p[:, N:]
        out["y"] = (_act(g, c["act"]) * u).bfloat16()
        if kind == "gated_fwd":
            return out
        g, u = (_dequantize(*_quantize(t, c["fmt"], c["group"]), N, c["group"]) for t in (g, u))
    else:
        g, u = (_stored(s[n], c["fmt"], c["group"]) for n in ("gate", "up"))
    a = _act(g, c["act"])
    dy = s["dy"].float() if kind == "gated_act_train" else torch.matmul(s["dz"].float(), s["w2"].float())
    dp = torch.cat([dy * u * _dact(g, c["act"]), dy * a], 1).bfloat16()
    hidden = (a * u).bfloat16()  # recomputed from what was kept
    out.update(dp=dp, hidden=hidden)
    if kind != "gated_dgrad":
        dp = dp.float()  # kept in bf16 between calls
        out.update(dx=torch.matmul(dp, w).bfloat16(), dw=torch.matmul(dp.t(), x).bfloat16())
    if kind == "gated_train":
        out["dw2"] = torch.matmul(s["dz"].float().t(), hidden.float()).bfloat16()
    return out


# ---- the framework's calls -----------------------------------------------------------

def _own(s):
    from learnable_scale_fake_gb300 import aqfq

    c = s["case"]
    kind = c["kind"]
    if kind.startswith("join"):
        aqfq.aqfq_block_norm_fwd(s["x"], s["f"], EPS, h=s["h"], y=s["y"], post=c["post"],
                                 gamma_post=s["gamma_post"], gate=s["gate"], alpha=s["alpha"],
                                 gamma_pre=s["gamma_pre"], rstd_post=s["rstd_post"],
                                 rstd_pre=s["rstd_pre"])
        names = ["h", "y", "rstd_post", "rstd_pre"]
        if kind == "join_train":
            aqfq.aqfq_block_norm_bwd(s["dy"], s["dh"], s["h"], s["f"], rstd_post=s["rstd_post"],
                                     rstd_pre=s["rstd_pre"], gamma_post=s["gamma_post"],
                                     gate=s["gate"], alpha=s["alpha"], gamma_pre=s["gamma_pre"],
                                     dx=s["dx"], df=s["df"], dgamma_post=s["dgamma_post"],
                                     dgate=s["dgate"], dgamma_pre=s["dgamma_pre"],
                                     workspace=s["workspace"])
            names += ["dx", "df", "dgamma_post", "dgate", "dgamma_pre"]
        return {n: s[n] for n in names if s[n] is not None}
    if kind == "rotary":
        aqfq.aqfq_rotary(s["q"], s["pos"], s["freqs"], s["yq"], k=s["k"], yk=s["yk"],
                         layout=aqfq.ROTARY_HALF if c["layout"] == "half" else aqfq.ROTARY_INTERLEAVED,
                         mscale=s["mscale"], transposed=c["transposed"])
        return {"q": s["yq"], "k": s["yk"]}
    act = {"relu": aqfq.ACT_RELU, "gelu": aqfq.ACT_GELU, "gelu_tanh": aqfq.ACT_GELU_TANH,
           "silu": aqfq.ACT_SILU}[c["act"]]
    ws = s["workspace"]
    if kind == "gated_fwd":
        aqfq.aqfq_gated_fwd(s["x"], s["w"], s["y"], act=act, workspace=ws)
        return {"y": s["y"]}
    fmt = aqfq.INT8 if c["fmt"] == "int8" else aqfq.FP8_E4M3
    gate, up = (aqfq.ckpt8(fmt, c["group"], *s[n]) for n in ("gate", "up"))
    out = {}
    if kind != "gated_dgrad":
        aqfq.aqfq_gated_fwd(s["x"], s["w"], s["y"], act=act, gate=gate, up=up, workspace=ws)
        out["y"] = s["y"]
    if kind == "gated_act_train":
        aqfq.aqfq_ckpt8_gated_bwd(gate, up, act, s["dy"], s["dp"], y=s["hidden"])
    else:
        aqfq.aqfq_gated_dgrad(s["dz"], s["w2"], s["dp"], gate, up, act=act, y=s["hidden"], workspace=ws)
    out.update(dp=s["dp"], hidden=s["hidden"])
    if kind != "gated_dgrad":
        aqfq.aqfq_linear_dgrad(s["dp"], s["w"], s["dx"], workspace=ws)
        aqfq.aqfq_linear_wgrad(s["dp"], s["x"], s["dw"], workspace=ws)
        out.update(dx=s["dx"], dw=s["dw"])
    if kind == "gated_train":
        aqfq.aqfq_linear_wgrad(s["dz"], s["hidden"], s["dw2"], workspace=ws)
        out["dw2"] = s["dw2"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    c = case
    kind = c["kind"]
    if kind.startswith("join"):
        R, C, b = c["rows"], c["cols"], 2 if c["dtype"] == "bf16" else 4
        n, vecs = R * C, 1 + c["post"] + c["gate"]
        by, fl = 4 * n * b + vecs * C * b + 4 * R * (1 + c["post"]), 10 * n  # x, f; h, y
        if kind == "join_train":  # dy, dh, h, f; dx, df
            by += 6 * n * b + vecs * C * (b + 4) + 4 * R * (1 + c["post"])
            fl += 20 * n
        return {"bytes": by, "flops": fl}
    if kind == "rotary":
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 8 * c["T"] + 4 * c["rot"],
                "flops": 3 * c["T"] * (c["Hq"] + c["Hk"]) * c["rot"]}
    M, N, K = c["M"], c["N"], c["K"]
    if kind == "gated_fwd":
        return {"bytes": 2 * (M * K + 2 * N * K + M * N), "flops": 4 * M * N * K}
    kept = 2 * (M * N + 4 * M * -(-N // c["group"]))  # gate and up in 8 bits
    D = c.get("D", 0)
    down = 2 * (M * D + D * N)  # dz, w2
    grad = kept + 2 * 3 * M * N  # what was kept; dp, the hidden activation
    if kind == "gated_dgrad":
        return {"bytes": down + grad, "flops": 2 * M * N * D}
    by = 2 * (M * K + 2 * N * K + M * N) + kept  # forward
    by += grad + (down + 2 * D * N if D else 2 * M * N)  # and dw2; or dy
    by += 2 * (2 * M * N + M * K + 2 * N * K)  # dp read again; dx, dw
    return {"bytes": by, "flops": (4 + 4 + 4) * M * N * K + 4 * M * N * D}


# ---- the definitions in 64 bits ------------------------------------------------------

def _kept64(x, fmt, group):
    """What an 8-bit checkpoint of x (float64 holding binary32 values) gives back.
    Scale and quotient are binary32 by definition (a quotient of two binary32
    values rounded first to 64 bits and then to 32 is the one rounded once); the
    grids are restated from their exponents and steps."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], group):
        t = x[:, lo:lo + group].float()
        top = t.abs().max(1, keepdim=True).values
        sc = (top.double() / QMAX[fmt]).float()
        v = (t.double() / sc.double()).float().double()
        v = torch.where(sc > 0, v, torch.zeros_like(v))
        if fmt == "int8":
            q = torch.round(v).clamp(-127, 127)
        else:
            e = torch.frexp(v).exponent - 1  # floor(log2 |v|)
            step = ((e.clamp(min=-6).long() - 3 + 1023) << 52).view(torch.float64)  # 2^(e - 3)
            q = (torch.round(v / step) * step).clamp(-448, 448)
        out[:, lo:lo + group] = (q * sc.double()).float().double()
    return out


def _act64(p, act):
    return {"relu": lambda: torch.where(p > 0, p, 0 * p), "gelu": lambda: p * torch.special.ndtr(p),
            "silu": lambda: p * torch.sigmoid(p),
            # 0.5 (1 + tanh u) = sigmoid(2 u)
            "gelu_tanh": lambda: p * torch.sigmoid(2 * math.sqrt(2 / math.pi)
                                                   * (p + 0.044715 * p ** 3))}[act]()


def _gated_grads(g, u, dy, act):
    """Gradients of act(g) u for g and u by automatic differentiation of the definition."""
    if act == "relu":
        return torch.where(g > 0, dy * u, torch.zeros_like(g)), dy * _act64(g, act)
    with torch.enable_grad():
        g, u = (t.detach().requires_grad_(True) for t in (g, u))
        return torch.autograd.grad((_act64(g, act) * u * dy).sum(), (g, u))


def _exact_join(s):
    c = s["case"]

    def rms(t):
        return 1.0 / torch.sqrt(torch.linalg.vector_norm(t, dim=1, keepdim=True) ** 2 / t.shape[1] + EPS)

    def rms_grad(t, r, d):  # of t r, r the reciprocal root mean square kept from the forward
        n = t * r
        return (d - n * torch.einsum("rc,rc->r", d, n)[:, None] / t.shape[1]) * r

    x, f, pre = s["x"].double(), s["f"].double(), s["gamma_pre"].double()
    coef = torch.full_like(pre, s["alpha"])
    if c["gate"]:
        coef = coef * s["gate"].double()
    rf = rms(f) if c["post"] else 1.0
    inner = coef * s["gamma_post"].double() if c["post"] else coef
    h = x + f * rf * inner
    rh = rms(h)
    out = {"h": h, "y": h * rh * pre, "rstd_pre": rh[:, 0]}
    if c["post"]:
        out["rstd_post"] = rf[:, 0]
    if c["kind"] == "join_fwd":
        return out
    kept, dy = h.to(s["x"].dtype).double(), s["dy"].double()
    dx = rms_grad(kept, rh, dy * pre) + s["dh"].double()
    out["dgamma_pre"] = torch.einsum("rc,rc->c", dy, kept * rh)
    if c["gate"]:
        out["dgate"] = s["alpha"] * torch.einsum(
            "rc,rc->c", dx, f * rf * (s["gamma_post"].double() if c["post"] else 1.0))
    if c["post"]:
        out["dgamma_post"] = coef * torch.einsum("rc,rc->c", dx, f * rf)
    out.update(dx=dx, df=rms_grad(f, rf, dx * inner) if c["post"] else dx * inner)
    return out


def _exact_rotary(s):
    """Each pair as a complex number times mscale exp(i angle)."""
    c, out = s["case"], {}
    turn = torch.polar(torch.full((c["T"], c["rot"] // 2), float(s["mscale"]), dtype=torch.float64,
                                  device="cuda"), torch.outer(s["pos"].double(), s["freqs"]))
    if c["transposed"]:
        turn = turn.conj()
    for name in ("q", "k"):
        x = s[name].double()
        z, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["layout"] == "half":
            z = z.unflatten(-1, (2, -1)).transpose(-1, -2)
        else:
            z = z.unflatten(-1, (-1, 2))
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None])
        if c["layout"] == "half":
            z = z.transpose(-1, -2)
        out[name] = torch.cat([z.flatten(-2), rest], -1)
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind.startswith("join"):
        return _exact_join(s)
    if kind == "rotary":
        return _exact_rotary(s)
    N, out = c["N"], {}
    if kind != "gated_dgrad":
        x, w = s["x"].double(), s["w"].double()
        g, u = x @ w[:N].T, x @ w[N:].T
        out["y"] = _act64(g, c["act"]) * u
        if kind == "gated_fwd":
            return out
        g, u = (_kept64(t.float().double(), c["fmt"], c["group"]) for t in (g, u))
    else:
        g, u = (_codes64(s[n], c["fmt"], c["group"]) for n in ("gate", "up"))
    dy = s["dy"].double() if kind == "gated_act_train" else s["dz"].double() @ s["w2"].double()
    dp = torch.cat(_gated_grads(g, u, dy, c["act"]), 1)
    hidden = _act64(g, c["act"]) * u
    out.update(dp=dp, hidden=hidden)
    if kind != "gated_dgrad":
        dp = dp.bfloat16().double()
        out.update(dx=dp @ w, dw=dp.T @ x)
    if kind == "gated_train":
        out["dw2"] = s["dz"].double().T @ hidden.bfloat16().double()
    return out


def _codes64(kept, fmt, group):
    q = kept[0].view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).double()
    col = torch.arange(q.shape[1], device=q.device) // group
    return (q * kept[1].double()[:, col]).float().double()
