"""Measured cases of the operators around the recurrence of a gated-delta-rule layer.

Three operators, each forward and backward:

  linear         y = residual + scale * act(x w^T + bias), the projections into and out of the
                 recurrence (plain, or with the pre-activation z kept for the backward)
  residual_norm  u = x (or its RMS norm times post_weight), h = residual + scale * gate * u,
                 y = RMS norm of h times weight: the norms on both sides of a block, its gate
                 and its residual scale in one pass
  gated_norm     y = RMS norm over each head of the recurrence's output o, times weight, times
                 act(gate)

`run` computes them in elementary torch operations in fp32 (own = False) or through the library's
entry points (own = True); `exact` evaluates the definitions in fp64, each written on its own.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"
BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}


# ------------------------------------------------------------------------------------------ cases

def _linear(name, T, K, N, dtype=BF16, y_dtype=None, bias=False, act="none", residual=False,
            scale=1.0, save_z=False):
    return dict(name=name, op="linear", T=T, K=K, N=N, dtype=dtype, y_dtype=y_dtype or dtype,
                bias=bias, act=act, residual=residual, scale=scale, save_z=save_z)


def _linear_bwd(name, T, K, N, dtype=BF16, bias=False, act="none", scale=1.0):
    return dict(name=name, op="linear_bwd", T=T, K=K, N=N, dtype=dtype, bias=bias, act=act,
                scale=scale)


def _norm(name, op, T, N, dtype=BF16, h_dtype=BF16, residual=True, post=False, gate="none",
          scale=1.0):
    return dict(name=name, op=op, T=T, N=N, dtype=dtype, h_dtype=h_dtype, residual=residual,
                post=post, gate=gate, scale=scale)


def _gated(name, op, T, H, D, o_dtype=F32, dtype=BF16, act="sigmoid"):
    return dict(name=name, op=op, T=T, H=H, D=D, o_dtype=o_dtype, dtype=dtype, act=act)


def listed():
    return [
        # one user's next token through the packed [Q | K | V] projection of 16 heads of 128:
        # the weight is the work, and the call's latency counts
        _linear("linear_one_token", 1, 2048, 6144),
        # the same projection of 32 heads for a decode batch of 256 sequences
        _linear("linear_decode_256", 256, 4096, 12288),
        # a ragged prompt batch (odd token count) through a GQA layer's projection (16 key and
        # 32 value heads) with bias and SiLU, the pre-activation kept for training
        _linear("linear_ragged_silu", 6731, 4096, 8192, bias=True, act="silu", save_z=True),
        # the output projection of a 2 x 16384 token prefill, added onto the residual stream
        _linear("linear_out_residual", 32768, 4096, 4096, residual=True, scale=0.5),
        # one training step's gradients of the packed projection on 4 x 4096 tokens
        _linear_bwd("linear_bwd_packed", 16384, 2048, 6144, bias=True),
        # a small fp32 model's layer, odd in every size, with an activation
        _linear_bwd("linear_bwd_odd_f32", 1003, 517, 1031, dtype=F32, bias=True, act="gelu",
                    scale=0.5),
        # the norms around a block in a decode step: norm of the block's output, per-channel
        # gate, fp32 residual stream, norm before the next block
        _norm("residual_norm_decode", "residual_norm", 256, 4096, h_dtype=F32, post=True,
              gate="channel", scale=0.5),
        # residual add and norm over a long prefill
        _norm("residual_norm_prefill", "residual_norm", 32768, 4096),
        # its gradients in training, with the norm after the block and a gate for each token
        _norm("residual_norm_bwd", "residual_norm_bwd", 16384, 2048, post=True, gate="token"),
        # the output norm of a decode batch
        _gated("gated_norm_decode", "gated_norm", 256, 32, 128),
        # the output norm of a long prefill
        _gated("gated_norm_prefill", "gated_norm", 32768, 32, 128),
        # its gradients in training
        _gated("gated_norm_bwd", "gated_norm_bwd", 16384, 16, 128, act="silu"),
    ]


_MAX_FLOPS = 2 * 32768 * 4096 * 4096
_MAX_F32_FLOPS = 2 * 8192 * 2048 * 2048
_MAX_BYTES = 32768 * 4096 * 8


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "linear_bwd", "residual_norm",
                     "residual_norm_bwd", "gated_norm", "gated_norm_bwd"])
    if op in ("linear", "linear_bwd"):
        dtype = BF16 if rng.random() < 0.75 else F32
        T = _log_int(rng, 1, 32768)
        K = _log_int(rng, 64, 8192)
        N = _log_int(rng, 16, 12288)
        if rng.random() < 0.7:                   # widths are mostly whole heads, tokens never are
            K = max(16, K // 16 * 16)
            N = max(16, N // 16 * 16)
        act = rng.choice(["none", "relu", "silu", "gelu", "sigmoid"])
        bias = rng.random() < 0.5
        scale = rng.choice([1.0, 0.5])
        cost = (2 if op == "linear" else 4) * K * N
        T = max(1, min(T, (_MAX_FLOPS if dtype == BF16 else _MAX_F32_FLOPS) // cost))
        if op == "linear":
            case = _linear(None, T, K, N, dtype=dtype, bias=bias, act=act,
                           y_dtype=rng.choice([dtype, F32]), residual=rng.random() < 0.5,
                           scale=scale, save_z=act != "none" and rng.random() < 0.5)
        else:
            case = _linear_bwd(None, T, K, N, dtype=dtype, bias=bias, act=act, scale=scale)
    elif op in ("residual_norm", "residual_norm_bwd"):
        N = _log_int(rng, 16, 16384)
        if rng.random() < 0.7:
            N = max(16, N // 16 * 16)
        case = _norm(None, op, _log_int(rng, 1, 32768), N, dtype=rng.choice([BF16, BF16, F32]),
                     h_dtype=rng.choice([BF16, F32]), residual=rng.random() < 0.8,
                     post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                     scale=rng.choice([1.0, 0.5]))
    else:
        D = rng.choice([16, 128, 128, 64, 256, 100, 37])
        H = rng.randint(1, 32)
        case = _gated(None, op, _log_int(rng, 1, 32768), H, D, o_dtype=rng.choice([F32, F32, BF16]),
                      dtype=rng.choice([BF16, BF16, F32]), act=rng.choice(["sigmoid", "silu"]))
    while work(case)["bytes"] > _MAX_BYTES:
        case["T"] = case["T"] * 3 // 4
    del case["name"]
    return case


# ----------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def normal(shape, dtype, std=1.0, mean=0.0):
        t = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
        return t.mul_(std).add_(mean).to(_DT[dtype])

    s = dict(case)
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        T, K, N, dt = case["T"], case["K"], case["N"], case["dtype"]
        # rows of a norm's output; weights of a trained or freshly initialised projection
        s["x"] = normal((T, K), dt)
        s["w"] = normal((N, K), dt, K ** -0.5)
        if op == "linear":
            s["bias_t"] = normal((N,), F32, 0.1) if case["bias"] else None
            s["residual_t"] = normal((T, N), dt) if case["residual"] else None
        else:
            s["z"] = normal((T, N), dt) if case["act"] != "none" else None
            s["dy"] = normal((T, N), dt, 1e-2)
    elif op in ("residual_norm", "residual_norm_bwd"):
        T, N, dt, hdt = case["T"], case["N"], case["dtype"], case["h_dtype"]
        s["x"] = normal((T, N), dt)
        s["weight"] = normal((N,), F32, 0.1, 1.0)
        s["post_weight"] = normal((N,), F32, 0.1, 1.0) if case["post"] else None
        s["gate_t"] = {"none": lambda: None, "channel": lambda: normal((N,), F32, 0.1, 0.5),
                       "token": lambda: normal((T, N), dt, 0.2, 0.5)}[case["gate"]]()
        if op == "residual_norm":
            s["residual_t"] = normal((T, N), hdt, 2.0) if case["residual"] else None
        else:
            s["h"] = normal((T, N), hdt, 2.0)      # the stored residual stream
            s["dy"] = normal((T, N), dt, 1e-2)
            s["dh"] = normal((T, N), hdt, 1e-2) if case["residual"] else None
    else:
        T, H, D = case["T"], case["H"], case["D"]
        s["o"] = normal((T, H, D), case["o_dtype"], 0.1)
        s["gate_t"] = normal((T, H, D), case["dtype"])
        s["weight"] = normal((D,), F32, 0.1, 1.0)
        if op == "gated_norm_bwd":
            s["dy"] = normal((T, H, D), case["dtype"], 1e-2)
    return s


# -------------------------------------------------------------------------------------- plain form

def _act(kind, z):
    if kind == "none":
        return z
    if kind == "relu":
        return z * (z > 0)
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))


def _act_grad(kind, z):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind in ("sigmoid", "silu"):
        p = 1 / (1 + torch.exp(-z))
        return p * (1 - p) if kind == "sigmoid" else p * (1 + z * (1 - p))
    return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))


def _rms(x):
    return 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias_t"] is not None:
        z = z + s["bias_t"]
    y = s["scale"] * _act(s["act"], z)
    if s["residual_t"] is not None:
        y = y + s["residual_t"].float()
    y = y.to(_DT[s["y_dtype"]])
    return (y, z.to(_DT[s["dtype"]])) if s["save_z"] else y


def _plain_linear_bwd(s):
    dz = s["scale"] * s["dy"].float()
    if s["act"] != "none":
        dz = dz * _act_grad(s["act"], s["z"].float())
    dt = _DT[s["dtype"]]
    out = ((dz @ s["w"].float()).to(dt), (dz.t() @ s["x"].float()).to(dt))
    return out + (dz.sum(0),) if s["bias"] else out


def _plain_residual_norm(s):
    u = s["x"].float()
    if s["post_weight"] is not None:
        u = u * _rms(u) * s["post_weight"]
    h = s["scale"] * u
    if s["gate_t"] is not None:
        h = h * s["gate_t"].float()
    if s["residual_t"] is not None:
        h = h + s["residual_t"].float()
    y = h * _rms(h) * s["weight"]
    return y.to(_DT[s["dtype"]]), h.to(_h_dtype(s))


def _h_dtype(s):
    return _DT[s["h_dtype"] if s["residual"] else s["dtype"]]


def _norm_grad(x, r, d):
    """Gradient of x * r, r the reciprocal RMS of x's rows, for an output gradient d."""
    n = x * r
    return r * (d - n * ((d * n).sum(-1, keepdim=True) / x.shape[-1]))


def _plain_residual_norm_bwd(s):
    h, dy, x = s["h"].float(), s["dy"].float(), s["x"].float()
    rh = _rms(h)
    dweight = (dy * h * rh).sum(0)
    dh = _norm_grad(h, rh, dy * s["weight"])
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    out = {"d_residual": dh.to(s["h"].dtype), "d_weight": dweight}
    du = s["scale"] * dh
    u = x
    if s["post_weight"] is not None:
        rx = _rms(x)
        u = x * rx * s["post_weight"]
    if s["gate_t"] is not None:
        dgate = du * u
        out["d_gate"] = dgate.sum(0) if s["gate"] == "channel" else dgate.to(s["gate_t"].dtype)
        du = du * s["gate_t"].float()
    if s["post_weight"] is not None:
        out["d_post_weight"] = (du * x * rx).sum(0)
        du = _norm_grad(x, rx, du * s["post_weight"])
    out["dx"] = du.to(s["x"].dtype)
    return out


def _plain_gated_norm(s):
    o = s["o"].float()
    return (o * _rms(o) * s["weight"] * _act(s["act"], s["gate_t"].float())).to(_DT[s["dtype"]])


def _plain_gated_norm_bwd(s):
    o, g, dy, w = s["o"].float(), s["gate_t"].float(), s["dy"].float(), s["weight"]
    r = _rms(o)
    n = o * r
    dn = dy * _act(s["act"], g)
    return (_norm_grad(o, r, dn * w).to(s["o"].dtype),
            (dy * n * w * _act_grad(s["act"], g)).to(s["gate_t"].dtype),
            (dn * n).sum((0, 1)))


# ------------------------------------------------------------------------------------ library calls

def _own_run(s):
    import gated_delta_rule_deltanet_gb300 as kda
    op = s["op"]
    if op == "linear":
        return kda.linear(s["x"], s["w"], s["bias_t"], activation=s["act"],
                          residual=s["residual_t"], scale=s["scale"], out_dtype=_DT[s["y_dtype"]],
                          save_pre_activation=s["save_z"])
    if op == "linear_bwd":
        out = kda.linear_bwd(s["x"], s["w"], s["dy"], activation=s["act"], pre_activation=s["z"],
                             scale=s["scale"], need_bias=s["bias"])
        return out if s["bias"] else out[:2]
    if op == "residual_norm":
        return kda.residual_norm(s["x"], s["weight"], residual=s["residual_t"],
                                 post_weight=s["post_weight"], gate=s["gate_t"], scale=s["scale"],
                                 eps=EPS)
    if op == "residual_norm_bwd":
        dx, dres, dw, dpw, dg = kda.residual_norm_bwd(
            s["x"], s["h"], s["weight"], s["dy"], s["dh"], post_weight=s["post_weight"],
            gate=s["gate_t"], scale=s["scale"], eps=EPS)
        out = {"d_residual": dres, "d_weight": dw}
        if dg is not None:
            out["d_gate"] = dg
        if dpw is not None:
            out["d_post_weight"] = dpw
        out["dx"] = dx
        return out
    if op == "gated_norm":
        return kda.gated_norm(s["o"], s["gate_t"], s["weight"], activation=s["act"], eps=EPS,
                              out_dtype=_DT[s["dtype"]])
    return kda.gated_norm_bwd(s["o"], s["gate_t"], s["weight"], s["dy"], activation=s["act"],
                              eps=EPS)


def run(state):
    if own:
        return _own_run(state)
    return {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd,
            "residual_norm": _plain_residual_norm, "residual_norm_bwd": _plain_residual_norm_bwd,
            "gated_norm": _plain_gated_norm, "gated_norm_bwd": _plain_gated_norm_bwd}[
                state["op"]](state)


# -------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        T, K, N, e = case["T"], case["K"], case["N"], _SIZE[case["dtype"]]
        if op == "linear":
            b = (T * K + N * K) * e + T * N * _SIZE[case["y_dtype"]]
            b += 4 * N * case["bias"] + T * N * e * (case["residual"] + case["save_z"])
            return {"bytes": b, "flops": 2 * T * K * N}
        b = 2 * (T * K + N * K) * e + T * N * e * (1 + (case["act"] != "none"))
        return {"bytes": b + 4 * N * case["bias"], "flops": 4 * T * K * N}
    if op in ("residual_norm", "residual_norm_bwd"):
        T, N, e, eh = case["T"], case["N"], _SIZE[case["dtype"]], _SIZE[case["h_dtype"]]
        post, token, channel = case["post"], case["gate"] == "token", case["gate"] == "channel"
        res = case["residual"]
        if op == "residual_norm":
            b = T * N * (2 * e + (2 * eh if res else e) + e * token) + 4 * N * (1 + post + channel)
            return {"bytes": b, "flops": T * N * (10 + 4 * post)}
        b = T * N * (3 * e + (2 + res) * eh + 2 * e * token) + 4 * N * (2 + 2 * post + 2 * channel)
        return {"bytes": b, "flops": T * N * (16 + 10 * post)}
    n, eo, e = case["T"] * case["H"] * case["D"], _SIZE[case["o_dtype"]], _SIZE[case["dtype"]]
    if op == "gated_norm":
        return {"bytes": n * (eo + 2 * e) + 4 * case["D"], "flops": n * 10}
    return {"bytes": n * (2 * eo + 3 * e) + 8 * case["D"], "flops": n * 25}


# ------------------------------------------------------------------------------------------- exact

def _sig64(v):
    return torch.sigmoid(v)


_ACT64 = {
    "none": (lambda v: v, lambda v: torch.ones_like(v)),
    "relu": (lambda v: v.clamp(min=0), lambda v: (v > 0).double()),
    "sigmoid": (_sig64, lambda v: _sig64(v) * _sig64(-v)),
    "silu": (lambda v: v * _sig64(v), lambda v: _sig64(v) + v * _sig64(v) * _sig64(-v)),
    "gelu": (lambda v: v * torch.special.ndtr(v),
             lambda v: torch.special.ndtr(v) + v * torch.exp(-v.square() / 2) / (2 * math.pi) ** 0.5),
}


def _unit64(v):
    """Rows divided by their RMS, and the factor."""
    f = (v.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return v * f, f


def _unit64_vjp(unit, f, d):
    return f * (d - unit * (unit * d).mean(-1, keepdim=True))


def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) else v for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op in ("linear", "linear_bwd"):
        act, dact = _ACT64[case["act"]]
        if op == "linear":
            z = torch.einsum("tk,nk->tn", s["x"], s["w"])
            z = z if s["bias_t"] is None else z + s["bias_t"][None]
            y = case["scale"] * act(z)
            y = y if s["residual_t"] is None else s["residual_t"] + y
            return (y, z) if case["save_z"] else y
        dz = case["scale"] * s["dy"]
        dz = dz if s["z"] is None else dz * dact(s["z"])
        dx = torch.einsum("tn,nk->tk", dz, s["w"])
        dw = torch.einsum("tn,tk->nk", dz, s["x"])
        return (dx, dw, dz.sum(0)) if case["bias"] else (dx, dw)
    if op in ("residual_norm", "residual_norm_bwd"):
        xu, xf = _unit64(s["x"])
        u = s["x"] if s["post_weight"] is None else xu * s["post_weight"]
        a = case["scale"] if s["gate_t"] is None else case["scale"] * s["gate_t"]
        if op == "residual_norm":
            h = a * u if s["residual_t"] is None else s["residual_t"] + a * u
            return _unit64(h)[0] * s["weight"], h
        hu, hf = _unit64(s["h"])
        dh = _unit64_vjp(hu, hf, s["dy"] * s["weight"])
        dh = dh if s["dh"] is None else dh + s["dh"]
        out = {"d_residual": dh, "d_weight": (s["dy"] * hu).sum(0)}
        if case["gate"] == "channel":
            out["d_gate"] = (case["scale"] * dh * u).sum(0)
        elif case["gate"] == "token":
            out["d_gate"] = case["scale"] * dh * u
        du = a * dh
        if s["post_weight"] is not None:
            out["d_post_weight"] = (du * xu).sum(0)
            du = _unit64_vjp(xu, xf, du * s["post_weight"])
        out["dx"] = du
        return out
    act, dact = _ACT64[case["act"]]
    ou, of = _unit64(s["o"])
    if op == "gated_norm":
        return ou * s["weight"] * act(s["gate_t"])
    dn = s["dy"] * act(s["gate_t"])
    return (_unit64_vjp(ou, of, dn * s["weight"]),
            s["dy"] * ou * s["weight"] * dact(s["gate_t"]), (dn * ou).sum((0, 1)))
