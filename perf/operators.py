"""The 16-bit operators of a transformer block around the quantised layers, as measured work.

Three operators, each in both directions:
  linear / linear_bwd   Y = act(X W^T + b) + R and its gradients
  norm / norm_bwd       layer norm with per-row-group scale and shift, and its gradients
  rope                  rotary positions with several axes (inverse = its gradient)
A case names its operator in "op".  `run` computes the plain form in 32 bits
with elementary torch operations, or, where `own` is true, calls the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one row through an adaLN modulation layer (width 1152, six vectors of scale, shift and gate)
        dict(name="linear 1 row, 1152 to 6912", op="linear", dtype="bf16", M=1, K=1152, N=6912,
             act="none", bias=True, residual=False, save=False),
        # a layer kept at 16 bits at the end of an MLP, with its residual: the largest product
        dict(name="linear 4608 x 12288 to 4608", op="linear", dtype="bf16", M=4608, K=12288, N=4608,
             act="none", bias=True, residual=True, save=False),
        # odd sizes of every kind, fp16, everything in the epilogue, the pre-activation kept for training
        dict(name="linear 333 x 1153 to 2307", op="linear", dtype="f16", M=333, K=1153, N=2307,
             act="gelu", bias=True, residual=True, save=True),
        # an MLP's first layer in training
        dict(name="linear back 4096, 1152 to 4608", op="linear_bwd", dtype="bf16", M=4096, K=1152,
             N=4608, act="gelu", bias=True),
        # a ragged batch in training, fp16
        dict(name="linear back 777, 1153 to 2305", op="linear_bwd", dtype="f16", M=777, K=1153, N=2305,
             act="silu", bias=True),
        # one token's norm: launch latency
        dict(name="norm 1 x 1152", op="norm", dtype="f32", params="f32", M=1, K=1152, groups=1,
             offset=0.0, affine=True, save=False),
        # modulated norm of four images of 4096 tokens, statistics kept for training
        dict(name="norm 16384 x 1152, 4 images", op="norm", dtype="bf16", params="bf16", M=16384,
             K=1152, groups=4, offset=1.0, affine=True, save=True),
        # a wide norm's gradients, fp32 parameters
        dict(name="norm back 4608 x 4608", op="norm_bwd", dtype="f16", params="f32", M=4608, K=4608,
             groups=1, offset=0.0, affine=True),
        # the modulated norm's gradients
        dict(name="norm back 16384 x 1152", op="norm_bwd", dtype="bf16", params="bf16", M=16384,
             K=1152, groups=4, offset=1.0, affine=True),
        # one token's queries and keys at a far position
        dict(name="rope 1 token", op="rope", dtype="bf16", T=1, H=64, D=128, pairs="8,28,28",
             pairing="interleaved", pad=4096, far=1 << 20, inverse=False),
        # image and text tokens: queries and keys in the rows of a fused QKV product
        dict(name="rope 4608 x 64 x 128", op="rope", dtype="bf16", T=4608, H=64, D=128,
             pairs="8,28,28", pairing="interleaved", pad=4096, far=64, inverse=False),
        # a video's tokens, head size 72 in halves, the gradient's direction
        dict(name="rope 16640 x 32 x 72 back", op="rope", dtype="f16", T=16640, H=32, D=72,
             pairs="12,12,12", pairing="halves", pad=0, far=4096, inverse=True),
    ]


def _log(rng, lo, hi):
    """An integer, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_MOST = 4608 * 12288 * 4608          # products of the largest listed case
_MOST_NORM = 16384 * 1152
_MOST_ROPE = 16640 * 32 * 72


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "norm", "norm_bwd", "rope"])
    if op in ("linear", "linear_bwd"):
        k, n = _log(rng, 64, 12288), _log(rng, 64, 12288)
        most = _MOST // (k * n) // (1 if op == "linear" else 2)
        c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), M=_log(rng, 1, min(16384, most)), K=k, N=n,
                 act=rng.choice(["none", "gelu", "silu"]), bias=rng.random() < 0.8)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        return c
    if op in ("norm", "norm_bwd"):
        k = _log(rng, 64, 12288)
        m = _log(rng, 1, _MOST_NORM // k)
        dtype = rng.choice(["bf16", "f16", "f32"])
        c = dict(op=op, dtype=dtype, params=rng.choice([dtype, "f32"]), M=m, K=k,
                 groups=min(m, rng.choice([1, 1, 2, 3, 4, 8])), offset=rng.choice([0.0, 1.0]),
                 affine=rng.random() < 0.85)
        if op == "norm":
            c.update(save=rng.random() < 0.5)
        return c
    axes = rng.choice([1, 2, 3])
    pairs = [rng.randint(1, 64 // axes) for _ in range(axes)]
    d = 2 * sum(pairs) + rng.choice([0, 0, 0, 8, 32])
    h = _log(rng, 1, 64)
    return dict(op="rope", dtype=rng.choice(["bf16", "f16", "f32"]), T=_log(rng, 1, _MOST_ROPE // (d * h) // 2),
                H=h, D=d, pairs=",".join(map(str, pairs)), pairing=rng.choice(["interleaved", "halves"]),
                pad=rng.choice([0, 0, 128, 1024]), far=_log(rng, 16, 1 << 22), inverse=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(g, m, k, dtype, scale=1.0, outliers=False):
    """[m, k] values in rows of a multiple of 16 bytes, as a view without the padding."""
    x = torch.randn((m, k), generator=g, device="cuda") * scale
    if outliers:         # one channel in a hundred is large, as in the activations of these models
        ch = torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")
        x[:, ch] *= 20.0
    out = _padded(m, k, dtype)
    out.copy_(x)
    return out


def _padded(m, k, dtype):
    return torch.empty((m, -(-k // 8) * 8), dtype=dtype, device="cuda")[:, :k]


def _group_rows(c):
    return -(-c["M"] // c["groups"])


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = _DT[c["dtype"]]
    s = dict(c)
    if c["op"] in ("linear", "linear_bwd"):
        M, K, N = c["M"], c["K"], c["N"]
        s["X"] = _rows(g, M, K, dt, outliers=True)
        s["W"] = _rows(g, N, K, dt, scale=0.02 if K > 256 else K ** -0.5)
        s["b"] = (torch.randn((N,), generator=g, device="cuda") * 0.1).to(dt) if c["bias"] else None
        if c["op"] == "linear":
            s["R"] = _rows(g, M, N, dt) if c["residual"] else None
            s["Y"] = _padded(M, N, dt)
            s["P"] = _padded(M, N, dt) if c["save"] else None
        else:
            s["dY"] = _rows(g, M, N, dt)
            s["P"] = None
            if c["act"] != "none":
                s["P"] = _rows(g, M, N, dt, scale=1.5)
            s["dX"], s["dW"] = _padded(M, K, dt), _padded(N, K, dt)
            s["db"] = torch.empty((N,), dtype=dt, device="cuda") if c["bias"] else None
            s["ws"] = None      # the library's workspace, made at the first call and kept
    elif c["op"] in ("norm", "norm_bwd"):
        M, K, G = c["M"], c["K"], c["groups"]
        pt = _DT[c["params"]]
        s["X"] = _rows(g, M, K, dt, outliers=True)
        s["X"] += torch.randn((M, 1), generator=g, device="cuda").to(dt)
        s["eps"] = 1e-6
        s["rows"] = _group_rows(c)
        used = -(-M // s["rows"])
        s["w"] = s["b"] = None
        if c["affine"]:
            s["w"] = _rows(g, used, K, pt, scale=0.2)
            s["w"] += 1.0 - c["offset"]
            s["b"] = _rows(g, used, K, pt, scale=0.2)
        if c["op"] == "norm":
            s["Y"] = _padded(M, K, dt)
            s["mean"] = torch.empty((M,), device="cuda") if c["save"] else None
            s["rstd"] = torch.empty((M,), device="cuda") if c["save"] else None
        else:
            s["dY"] = _rows(g, M, K, dt)
            x = s["X"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(1) + s["eps"]).rsqrt().float()
            s["dX"] = _padded(M, K, dt)
            s["dw"] = _padded(used, K, pt) if c["affine"] else None
            s["db"] = _padded(used, K, pt) if c["affine"] else None
            s["ws"] = None
    else:
        T, H, D = c["T"], c["H"], c["D"]
        pairs = [int(p) for p in c["pairs"].split(",")]
        row = -(-(H * D + c["pad"]) // 8) * 8
        buf = torch.randn((T, row), generator=g, device="cuda").to(dt)
        s["X"] = buf[:, :H * D].unflatten(1, (H, D))
        s["out"] = torch.empty((T, -(-(H * D) // 8) * 8), dtype=dt, device="cuda")[:, :H * D].unflatten(1, (H, D))
        s["pos"] = torch.randint(0, c["far"], (T, len(pairs)), generator=g, device="cuda", dtype=torch.int32)
        s["freq"] = [10000.0 ** (-i / p) for p in pairs for i in range(p)]
        s["f64"] = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
        s["axis"] = torch.tensor([a for a, p in enumerate(pairs) for _ in range(p)], device="cuda")
        s["n_pairs"] = pairs
        s["plan"] = None        # the library's plan, made at the first call and kept
    return s


# --------------------------------------------------------------- plain forms
def _act(y, act):
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y * torch.sigmoid(y) if act == "silu" else y


def _act_grad(p, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(p * math.sqrt(0.5))) + p * torch.exp(-0.5 * p * p) / math.sqrt(2 * math.pi)
    q = torch.sigmoid(p)
    return q * (1.0 + p * (1.0 - q))


def _linear(s):
    p = s["X"].float() @ s["W"].float().t()
    if s["b"] is not None:
        p = p + s["b"].float()
    y = _act(p, s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    dt = s["X"].dtype
    return (y.to(dt), p.to(dt)) if s["save"] else y.to(dt)


def _linear_bwd(s):
    d, dt = s["dY"].float(), s["X"].dtype
    if s["act"] != "none":
        d = d * _act_grad(s["P"].float(), s["act"])
    out = [(d @ s["W"].float()).to(dt), (d.t() @ s["X"].float()).to(dt)]
    return out + [d.sum(0).to(dt)] if s["bias"] else out


def _per_row(p, s):
    """A parameter's row for each row of X."""
    return p.float().repeat_interleave(s["rows"], 0)[:s["M"]]


def _norm(s):
    x = s["X"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + s["eps"])
    y = d * rstd
    if s["affine"]:
        y = y * (_per_row(s["w"], s) + s["offset"]) + _per_row(s["b"], s)
    y = y.to(s["X"].dtype)
    return (y, mean[:, 0], rstd[:, 0]) if s["save"] else y


def _group_sum(v, s):
    """[M, K] summed over each group's rows."""
    short = -v.shape[0] % s["rows"]
    if short:
        v = torch.cat([v, v.new_zeros((short, v.shape[1]))])
    return v.view(-1, s["rows"], v.shape[1]).sum(1)


def _norm_bwd(s):
    dy, rstd = s["dY"].float(), s["rstd"][:, None]
    xhat = (s["X"].float() - s["mean"][:, None]) * rstd
    g = dy * (_per_row(s["w"], s) + s["offset"]) if s["affine"] else dy
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    out = [dx.to(s["X"].dtype)]
    if s["affine"]:
        out += [_group_sum(dy * xhat, s).to(s["w"].dtype), _group_sum(dy, s).to(s["b"].dtype)]
    return out


def _rope(s):
    angle = s["pos"].double()[:, s["axis"]] * s["f64"]           # far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if s["inverse"]:
        sin = -sin
    x, n = s["X"].float(), s["f64"].numel()
    y = x.clone()
    if s["pairing"] == "interleaved":
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * cos - b * sin, a * sin + b * cos
    return y.to(s["X"].dtype)


# ------------------------------------------------------- the library's calls
def _own(s):
    import w4a4_quantized_gemm_smooth_b200 as S
    op = s["op"]
    if op in ("linear", "linear_bwd"):
        epi = {"none": S.EPI_NONE, "gelu": S.EPI_GELU, "silu": S.EPI_SILU}[s["act"]]
    if op == "linear":
        S.svdq_linear16(s["X"], s["W"], s["Y"], bias=s["b"], residual=s["R"], epilogue=epi, preact=s["P"])
        return (s["Y"], s["P"]) if s["save"] else s["Y"]
    if op == "linear_bwd":
        if s["ws"] is None:
            n = S.svdq_linear16_backward_workspace(s["M"], s["K"], s["N"], epi)
            s["ws"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
        S.svdq_linear16_backward(s["dY"], s["X"], s["W"], s["P"], s["dX"], s["dW"], s["db"], s["ws"], epilogue=epi)
        out = [s["dX"], s["dW"]]
        return out + [s["db"]] if s["bias"] else out
    if op == "norm":
        S.svdq_layer_norm(s["X"], s["Y"], s["w"], s["b"], eps=s["eps"], weight_offset=s["offset"],
                          rows_per_group=s["rows"], mean=s["mean"], rstd=s["rstd"])
        return (s["Y"], s["mean"], s["rstd"]) if s["save"] else s["Y"]
    if op == "norm_bwd":
        if s["ws"] is None:
            n = S.svdq_layer_norm_backward_workspace(s["M"], s["K"], s["rows"])
            s["ws"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
        S.svdq_layer_norm_backward(s["dY"], s["X"], s["mean"], s["rstd"], s["dX"], s["w"],
                                   weight_offset=s["offset"], rows_per_group=s["rows"], dweight=s["dw"],
                                   dbias=s["db"], workspace=s["ws"])
        return [s["dX"], s["dw"], s["db"]] if s["affine"] else [s["dX"]]
    if s["plan"] is None:
        pairing = S.ROPE_INTERLEAVED if s["pairing"] == "interleaved" else S.ROPE_HALVES
        s["plan"] = S.svdq_rope_create(s["n_pairs"], s["freq"], pairing)
    S.svdq_rope(s["plan"], s["pos"], s["X"], s["out"], inverse=s["inverse"])
    return s["out"]


_PLAIN = {"linear": _linear, "linear_bwd": _linear_bwd, "norm": _norm, "norm_bwd": _norm_bwd, "rope": _rope}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- the work
def work(case):
    c = case
    e = {"bf16": 2, "f16": 2, "f32": 4}
    b = e[c["dtype"]]
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        n = M * K + N * K + M * N * (1 + c["residual"] + c["save"]) + N * c["bias"]
        return {"bytes": b * n, "flops": 2 * M * N * K}
    if c["op"] == "linear_bwd":
        M, K, N = c["M"], c["K"], c["N"]
        n = M * N * (1 + (c["act"] != "none")) + 2 * M * K + 2 * N * K + N * c["bias"]
        return {"bytes": b * n, "flops": 4 * M * N * K}
    if c["op"] in ("norm", "norm_bwd"):
        M, K = c["M"], c["K"]
        used = -(-M // _group_rows(c)) if c["affine"] else 0
        if c["op"] == "norm":
            return {"bytes": 2 * b * M * K + 2 * used * K * e[c["params"]] + 8 * M * c["save"], "flops": 8 * M * K}
        return {"bytes": 3 * b * M * K + 3 * used * K * e[c["params"]] + 8 * M, "flops": 14 * M * K}
    n = c["T"] * c["H"] * c["D"]
    return {"bytes": 2 * b * n + 4 * c["T"] * len(c["pairs"].split(",")), "flops": 3 * n}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if s["op"] == "linear":
        p = torch.einsum("mk,nk->mn", s["X"].to(d), s["W"].to(d))
        p += 0 if s["b"] is None else s["b"].to(d)
        y = {"none": lambda v: v, "gelu": lambda v: v * torch.special.ndtr(v),
             "silu": lambda v: v / (1 + torch.exp(-v))}[s["act"]](p)
        if s["R"] is not None:
            y = y + s["R"].to(d)
        return (y, p) if s["save"] else y
    if s["op"] == "linear_bwd":
        dp = s["dY"].to(d)
        if s["act"] != "none":
            with torch.enable_grad():
                p = s["P"].to(d).requires_grad_()
                y = p * torch.special.ndtr(p) if s["act"] == "gelu" else p / (1 + torch.exp(-p))
                dp, = torch.autograd.grad(y, p, dp)
        dx = torch.einsum("mn,nk->mk", dp, s["W"].to(d))
        dw = torch.einsum("mn,mk->nk", dp, s["X"].to(d))
        return [dx, dw, torch.einsum("mn->n", dp)] if s["bias"] else [dx, dw]
    if s["op"] in ("norm", "norm_bwd"):
        row = torch.arange(s["M"], device="cuda") // s["rows"]
        x = s["X"].to(d)
        w = s["w"].to(d)[row] + s["offset"] if s["affine"] else torch.ones((), dtype=d, device="cuda")
        if s["op"] == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + s["eps"]) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None] * w + (s["b"].to(d)[row] if s["affine"] else 0)
            return (y, mean, rstd) if s["save"] else y
        # the gradients for the given statistics, each a projection of w dy
        dy, r = s["dY"].to(d), s["rstd"].to(d)[:, None]
        h = (x - s["mean"].to(d)[:, None]) * r
        t = dy * w
        dx = t - torch.einsum("mk->m", t)[:, None] / s["K"] - h * torch.einsum("mk,mk->m", t, h)[:, None] / s["K"]
        if not s["affine"]:
            return [r * dx]
        zero = torch.zeros(s["w"].shape, dtype=d, device="cuda")
        return [r * dx, zero.index_add(0, row, dy * h), zero.index_add(0, row, dy)]
    # a pair as a complex number, turned by its angle
    n = len(s["freq"])
    x = s["X"].to(d)
    pos = torch.repeat_interleave(s["pos"].to(d), torch.tensor(s["n_pairs"], device="cuda"), 1)
    turn = torch.polar(torch.ones((), dtype=d, device="cuda"), pos * s["f64"] * (-1.0 if s["inverse"] else 1.0))
    if s["pairing"] == "interleaved":
        z = torch.view_as_complex(x[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * turn[:, None]
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :n], x[..., n:2 * n]) * turn[:, None]
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)
