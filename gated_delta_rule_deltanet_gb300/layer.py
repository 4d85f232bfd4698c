"""Torch-facing binding of the layer around the recurrence: the projections, the norms on both
sides of a block and the output norm with its gate (kda_linear_*, kda_residual_norm_*,
kda_gated_norm_*).  Argument marshalling only, as in `kda.py`.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import KdaError, KdaLinearParams, KdaNormParams
from .kda import _QKV_DTYPES, _workspace

_ACTIVATIONS = {"none": _lib.KDA_ACT_NONE, "relu": _lib.KDA_ACT_RELU, "silu": _lib.KDA_ACT_SILU,
                "gelu": _lib.KDA_ACT_GELU, "sigmoid": _lib.KDA_ACT_SIGMOID}
_NORM_GATES = ("sigmoid", "silu", "none")


# A call's checks and parameter record depend only on its tensors' shapes, strides, types and
# devices and on its scalars, so they are made once for each combination of those (`_sig`) and kept:
# a decode step repeats the same few thousands of times, and the checks would cost more than its
# kernels.  Nothing is kept by a tensor's address or contents: a scalar given as a tensor is read
# on each call.
_PLANS: dict = {}
_MAX_PLANS = 4096


class _Plan:
    __slots__ = ("fn", "params", "ref", "device", "index", "nbytes", "shape", "dtype", "dtype2", "pairs",
                 "pools", "reach")

    def __init__(self, name, params, device, nbytes=0, shape=None, dtype=None, dtype2=None):
        self.fn = getattr(_lib.load(), name)
        self.params = params
        self.ref = ctypes.byref(params)
        self.device = device
        self.index = device.index
        self.nbytes = nbytes
        self.shape = shape
        self.dtype = dtype
        self.dtype2 = dtype2
        self.pairs = ()


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _sig16(t):
    """The same with the address's place within 16 bytes, where a copy depends on it."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device(), t.data_ptr() & 15)


def _keep(key, plan):
    if len(_PLANS) >= _MAX_PLANS:
        _PLANS.clear()
    _PLANS[key] = plan
    return plan


def _device(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def _p(t):
    return None if t is None else t.data_ptr()


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the handle of the current stream without building a Stream object (2 us a call), and the current
# device without the check for initialisation, where torch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(stream, t):
    """With `stream=`, the whole call runs with that stream current, so that the outputs and the
    workspace it allocates belong to the stream that uses them."""
    if stream.device != t.device:
        raise ValueError("the stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _call(plan, *args):
    """Calls the plan's entry point on the current stream of its device, that device current."""
    index = plan.index
    if _current_device() == index:
        st = plan.fn(plan.ref, *args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = plan.fn(plan.ref, *args, _raw_stream(index))
    if st != _lib.KDA_OK:
        raise KdaError(st, plan.fn.__name__)


def _space(plan, workspace):
    """The call's workspace: (tensor or None, its address or None, its bytes)."""
    need = plan.nbytes
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=plan.device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != plan.device:
        raise ValueError("all tensors must be on the same device")
    _workspace(need, workspace, plan.device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _rows(t, shape, dtypes, name):
    """Checks a [T, C] array with dense rows; returns the elements between rows (0: one row or
    dense)."""
    if t.dim() != 2 or t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must be {list(shape)} {' / '.join(str(d) for d in dtypes)}")
    if shape[0] > 1 and shape[1] > 0:
        if shape[1] > 1 and t.stride(1) != 1 or t.stride(0) < shape[1]:
            raise ValueError(f"{name} must have dense rows")
        return t.stride(0)
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows")
    return 0


def _runs(t):
    """How the elements of t lie: (number, bytes apart) of its dimensions from the outermost on, joined where they can
    be, and the bytes of a dense run."""
    width, dims = t.element_size(), []
    run = width
    for apart, n in sorted((s * width, n) for s, n in zip(t.stride(), t.shape) if n > 1 and s > 0):
        if not dims and apart == run:
            run *= n
        elif dims and apart == dims[-1][0] * dims[-1][1]:
            dims[-1] = (n * dims[-1][0], dims[-1][1])
        else:
            dims.append((n, apart))
    return dims[::-1], run


def _reach(outer, run):
    return run + sum((n - 1) * s for n, s in outer)


def _runs_meet(a, outer_a, run_a, b, outer_b, run_b):
    ends_a, ends_b = _reach(outer_a, run_a), _reach(outer_b, run_b)
    if a + ends_a <= b or b + ends_b <= a:
        return False
    if not outer_a and not outer_b:
        return True
    if outer_a and outer_b and outer_a[0][1] == outer_b[0][1]:
        (n, s), (m, _) = outer_a[0], outer_b[0]
        inner_a, inner_b = ends_a - (n - 1) * s, ends_b - (m - 1) * s
        if inner_a <= s and inner_b <= s:
            # blocks in step, as of two columns of one packed array: b's block i lies `shift` behind a's block i + k
            # or, the step before, i + k + 1
            k, shift = divmod(b - a, s)
            return any(-m < i < n and _runs_meet(0, outer_a[1:], run_a, d, outer_b[1:], run_b)
                       for i, d in ((k, shift), (k + 1, shift - s)))
    if not outer_a or outer_b and ends_a < ends_b:
        a, outer_a, run_a, ends_a, b, outer_b, run_b, ends_b = b, outer_b, run_b, ends_b, a, outer_a, run_a, ends_a
    n, s = outer_a[0]
    inner = ends_a - (n - 1) * s
    return any(_runs_meet(a + i * s, outer_a[1:], run_a, b, outer_b, run_b)
               for i in range(max(0, (b - a - inner) // s + 1), min(n - 1, (b + ends_b - 1 - a) // s) + 1))


def _pairs(tensors, *which):
    """What a plan keeps to tell whether an output shares memory with another tensor, whose blocks would write what others
    still read.  `which`: (name of the output, its place among `tensors`, the other's), and True where the output may
    be the other one itself."""
    pairs = []
    for name, i, j, *itself in which:
        x, y = tensors[i], tensors[j]
        if x is not None and y is not None and x.numel() and y.numel():
            a, b = _runs(x), _runs(y)
            # bytes between the rows where both are rows that far apart, as two columns of one packed array
            step = a[0][0][1] if len(a[0]) == len(b[0]) == 1 and a[0][0][1] == b[0][0][1] else 0
            pairs.append((i, _reach(*a), j, _reach(*b), name, a, b, step, bool(itself) and a == b))
    return tuple(pairs)


def _apart(pairs, *tensors):
    for i, ends_a, j, ends_b, name, runs_a, runs_b, step, itself in pairs:
        a, b = tensors[i].data_ptr(), tensors[j].data_ptr()
        if a >= b + ends_b or b >= a + ends_a or itself and a == b:
            continue
        if step and runs_a[1] <= (b - a) % step <= step - runs_b[1]:
            continue
        if _runs_meet(a, *runs_a, b, *runs_b):
            raise ValueError(f"{name} must have memory of its own" + (" or be its input itself" if itself else ""))
    return pairs


def _dense(t, shape, dtype, name):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}")


def _linear_params(x, weight, activation, scale, y_dtype, flags):
    if x.dim() != 2 or x.dtype not in _QKV_DTYPES:
        raise ValueError("x must be [T, K] float32 or bfloat16")
    if weight.dim() != 2:
        raise ValueError("weight must be [N, K]")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(_ACTIVATIONS)}")
    if y_dtype not in _QKV_DTYPES:
        raise ValueError("the output dtype must be float32 or bfloat16")
    (T, K), N = x.shape, weight.shape[0]
    dt = _QKV_DTYPES[x.dtype]
    return KdaLinearParams(
        tokens=T, in_features=K, out_features=N, dtype=dt, y_dtype=_QKV_DTYPES[y_dtype],
        residual_dtype=dt, dw_dtype=dt, activation=_ACTIVATIONS[activation], scale=scale,
        x_row_stride=_rows(x, (T, K), (x.dtype,), "x"),
        w_row_stride=_rows(weight, (N, K), (x.dtype,), "weight"),
        flags=flags | _unaligned(x, _lib.KDA_FLAG_UNALIGNED_X)
        | _unaligned(weight, _lib.KDA_FLAG_UNALIGNED_W))


def _unaligned(t, flag):
    return flag if t.data_ptr() % 16 else 0


def _bytes(name, p, flag, dev):
    """A workspace size, asked for with the tensors' device current (it depends on its SMs)."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(dev):
        st = getattr(_lib.load(), name)(ctypes.byref(p), flag, ctypes.byref(n))
    if st != _lib.KDA_OK:
        raise KdaError(st, name)
    return n.value


def _linear_plan(key, p, backward, dev, shape, y_dtype, dw_dtype=None):
    nbytes = _bytes("kda_linear_workspace_size", p, backward, dev)
    return _keep(key, _Plan("kda_linear_bwd" if backward else "kda_linear_fwd", p, dev, nbytes, shape,
                            y_dtype, dw_dtype))


def _plan_linear(key, x, weight, bias, activation, residual, scale, out_dtype, out, cuda_cores):
    dev = _device(x, weight, bias, residual, out)
    y_dtype = out.dtype if out is not None else (out_dtype or x.dtype)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out does not have out_dtype")
    p = _linear_params(x, weight, activation, scale, y_dtype,
                       _lib.KDA_FLAG_CUDA_CORES if cuda_cores else 0)
    T, N = x.shape[0], weight.shape[0]
    if bias is not None:
        _dense(bias, (N,), torch.float32, "bias")
    if residual is not None:
        p.residual_row_stride = _rows(residual, (T, N), tuple(_QKV_DTYPES), "residual")
        p.residual_dtype = _QKV_DTYPES[residual.dtype]
    if out is not None:
        p.y_row_stride = _rows(out, (T, N), (y_dtype,), "out")
    return _linear_plan(key, p, 0, dev, (T, N), y_dtype)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           activation: str = "none", residual: Optional[torch.Tensor] = None, scale: float = 1.0,
           out_dtype: Optional[torch.dtype] = None, save_pre_activation: bool = False,
           cuda_cores: bool = False, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None):
    """Projection with its epilogue (kda_linear_fwd): residual + scale * act(x weight^T + bias).

    x [T, K] and weight [N, K] in one dtype, rows dense with any stride (tensor cores with fp32
    sums; float32 as three bfloat16 parts; `cuda_cores=True`: fp32 CUDA cores); bias [N] float32;
    residual [T, N] float32 or bfloat16.  `activation`: none, relu, silu, gelu (erf form) or
    sigmoid.  Returns y [T, N] in `out_dtype` (default x's), or (y, z) with
    `save_pre_activation`, z [T, N] in x's dtype being what `linear_bwd` needs as
    `pre_activation`.  `out` may be `residual` itself; it shares no memory with x or weight.
    """
    if stream is not None:
        with _on(stream, x):
            return linear(x, weight, bias, activation=activation, residual=residual, scale=scale,
                          out_dtype=out_dtype, save_pre_activation=save_pre_activation,
                          cuda_cores=cuda_cores, out=out, workspace=workspace)
    scale = float(scale)
    key = ("linear", x.shape, x.stride(), x.dtype, x.get_device(), x.data_ptr() & 15, _sig16(weight),
           _sig(bias), activation, _sig(residual), scale, out_dtype, _sig(out), cuda_cores)
    plan = _PLANS.get(key)
    if plan is None:
        pairs = _apart(_pairs((out, x, weight), ("out", 0, 1), ("out", 0, 2)), out, x, weight)
        plan = _plan_linear(key, x, weight, bias, activation, residual, scale, out_dtype, out,
                            cuda_cores)
        plan.pairs = pairs
    elif plan.pairs:
        _apart(plan.pairs, out, x, weight)
    if out is None:
        out = torch.empty(plan.shape, dtype=plan.dtype, device=plan.device)
    z = torch.empty(plan.shape, dtype=x.dtype, device=plan.device) if save_pre_activation else None
    space, address, nbytes = _space(plan, workspace)
    _call(plan, x.data_ptr(), weight.data_ptr(), _p(bias), _p(residual),
          out.data_ptr(), _p(z), address, nbytes)
    return (out, z) if save_pre_activation else out


def _plan_linear_bwd(key, x, weight, d_y, activation, pre_activation, scale, dw_dtype, cuda_cores):
    dev = _device(x, weight, d_y, pre_activation)
    if d_y.dtype not in _QKV_DTYPES:
        raise ValueError("d_y must be float32 or bfloat16")
    p = _linear_params(x, weight, activation, scale, d_y.dtype,
                       _lib.KDA_FLAG_CUDA_CORES if cuda_cores else 0)
    T, N = x.shape[0], weight.shape[0]
    p.y_row_stride = _rows(d_y, (T, N), (d_y.dtype,), "d_y")
    p.flags |= _unaligned(d_y, _lib.KDA_FLAG_UNALIGNED_DY)
    if activation != "none":
        if pre_activation is None:
            raise ValueError("an activation's gradient needs pre_activation")
        _dense(pre_activation, (T, N), x.dtype, "pre_activation")
    dw_dtype = dw_dtype or x.dtype
    if dw_dtype not in _QKV_DTYPES:
        raise ValueError("dw_dtype must be float32 or bfloat16")
    p.dw_dtype = _QKV_DTYPES[dw_dtype]
    return _linear_plan(key, p, 1, dev, (T, N), d_y.dtype, dw_dtype)


def linear_bwd(x: torch.Tensor, weight: torch.Tensor, d_y: torch.Tensor, *,
               activation: str = "none", pre_activation: Optional[torch.Tensor] = None,
               scale: float = 1.0, need_dx: bool = True, need_dw: bool = True,
               need_bias: bool = False, dw_dtype: Optional[torch.dtype] = None,
               cuda_cores: bool = False, workspace: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Backward of `linear` (kda_linear_bwd).  d_y [T, N] float32 or bfloat16; `pre_activation`
    as `linear` returned it (needed with an activation).  With an activation or a float32 d_y,
    bfloat16 operands round act'(z) d_y to bfloat16 before the two products.  Returns (dx [T, K]
    in x's dtype, dw [N, K] in `dw_dtype` (default x's), dbias [N] float32), None for those not
    needed.
    The residual's gradient is d_y itself."""
    if stream is not None:
        with _on(stream, x):
            return linear_bwd(x, weight, d_y, activation=activation, pre_activation=pre_activation,
                              scale=scale, need_dx=need_dx, need_dw=need_dw, need_bias=need_bias,
                              dw_dtype=dw_dtype, cuda_cores=cuda_cores, workspace=workspace)
    if activation == "none":
        pre_activation = None
    scale = float(scale)
    key = ("linear_bwd", _sig16(x), _sig16(weight), _sig16(d_y), activation, _sig(pre_activation),
           scale, dw_dtype, cuda_cores)
    plan = _PLANS.get(key)
    if plan is None:
        plan = _plan_linear_bwd(key, x, weight, d_y, activation, pre_activation, scale, dw_dtype,
                                cuda_cores)
    dev = plan.device
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need_dx else None
    dw = torch.empty(weight.shape, dtype=plan.dtype2, device=dev) if need_dw else None
    dbias = torch.empty(plan.shape[1:], dtype=torch.float32, device=dev) if need_bias else None
    space, address, nbytes = _space(plan, workspace)
    _call(plan, x.data_ptr(), weight.data_ptr(), _p(pre_activation),
          d_y.data_ptr(), _p(dx), _p(dw), _p(dbias), address, nbytes)
    return dx, dw, dbias


# ----------------------------------------------------------------------------------------- norms

def _norm_gate(gate, x, p, N):
    if gate is None:
        return
    if gate.dim() == 1:
        _dense(gate, (N,), torch.float32, "a per-channel gate")
    else:
        p.gate_per_token = 1
        p.gate_row_stride = _rows(gate, tuple(x.shape), (x.dtype,), "a per-token gate")


def _residual_params(x, h_dtype, scale, eps):
    if x.dim() != 2 or x.dtype not in _QKV_DTYPES or not x.is_contiguous():
        raise ValueError("x must be contiguous [T, N] float32 or bfloat16")
    dt = _QKV_DTYPES[x.dtype]
    return KdaNormParams(tokens=x.shape[0], features=x.shape[1], x_dtype=dt,
                         h_dtype=_QKV_DTYPES[h_dtype], y_dtype=dt, eps=eps, scale=scale)


def _plan_residual_norm(key, x, weight, residual, post_weight, gate, scale, eps, out, h_out):
    dev = _device(x, weight, residual, post_weight, gate, out, h_out)
    h_dtype = residual.dtype if residual is not None else x.dtype
    if h_dtype not in _QKV_DTYPES:
        raise ValueError("residual must be float32 or bfloat16")
    p = _residual_params(x, h_dtype, scale, eps)
    shape, N = x.shape, x.shape[1]
    if residual is not None:
        _dense(residual, shape, h_dtype, "residual")
    for name, t in (("weight", weight), ("post_weight", post_weight)):
        if t is not None:
            _dense(t, (N,), torch.float32, name)
    _norm_gate(gate, x, p, N)
    if h_out is not None:
        _dense(h_out, shape, h_dtype, "h_out")
    if out is not None:
        if weight is None:
            raise ValueError("out needs a weight")
        _dense(out, shape, x.dtype, "out")
    return _keep(key, _Plan("kda_residual_norm_fwd", p, dev, 0, shape, h_dtype))


def residual_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                  residual: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  scale: float = 1.0, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
                  h_out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None):
    """The norms around a block in one pass (kda_residual_norm_fwd).  With
    rms(a) = a / sqrt(mean(a^2) + eps) over each row:

        u = rms(x) * post_weight (x without one);  h = residual + scale * gate * u;
        y = rms(h) * weight

    x [T, N]; residual [T, N] (float32 or bfloat16: h's dtype); gate [N] float32 or [T, N] in x's
    dtype (row stride free); weights [N] float32.  Returns (y in x's dtype, or None without
    `weight`; h in the residual's dtype, x's without one).  `h_out` may be `residual`.
    """
    if stream is not None:
        with _on(stream, x):
            return residual_norm(x, weight, residual=residual, post_weight=post_weight, gate=gate,
                                 scale=scale, eps=eps, out=out, h_out=h_out)
    scale, eps = float(scale), float(eps)
    key = ("residual_norm", _sig(x), _sig(weight), _sig(residual), _sig(post_weight), _sig(gate),
           scale, eps, _sig(out), _sig(h_out))
    plan = _PLANS.get(key)
    if plan is None:
        pairs = _apart(_pairs((out, h_out), ("out", 0, 1)), out, h_out)
        plan = _plan_residual_norm(key, x, weight, residual, post_weight, gate, scale, eps, out,
                                   h_out)
        plan.pairs = pairs
    elif plan.pairs:
        _apart(plan.pairs, out, h_out)
    if h_out is None:
        h_out = torch.empty(plan.shape, dtype=plan.dtype, device=plan.device)
    if out is None and weight is not None:
        out = torch.empty_like(x)
    _call(plan, x.data_ptr(), _p(residual), _p(gate), _p(post_weight),
          _p(weight), h_out.data_ptr(), _p(out))
    return out, h_out


def _plan_residual_norm_bwd(key, x, h, weight, d_y, d_h, post_weight, gate, scale, eps):
    dev = _device(x, h, weight, d_y, d_h, post_weight, gate)
    if h.dtype not in _QKV_DTYPES:
        raise ValueError("h must be float32 or bfloat16")
    p = _residual_params(x, h.dtype, scale, eps)
    shape, N = x.shape, x.shape[1]
    _dense(h, shape, h.dtype, "h")
    if (weight is None) != (d_y is None):
        raise ValueError("d_y and weight come together")
    if d_y is None and d_h is None:
        raise ValueError("one of d_y and d_h is needed")
    if d_y is not None:
        _dense(d_y, shape, x.dtype, "d_y")
    if d_h is not None:
        _dense(d_h, shape, h.dtype, "d_h")
    for name, t in (("weight", weight), ("post_weight", post_weight)):
        if t is not None:
            _dense(t, (N,), torch.float32, name)
    _norm_gate(gate, x, p, N)
    nbytes = _bytes("kda_norm_workspace_size", p, 0, dev)
    return _keep(key, _Plan("kda_residual_norm_bwd", p, dev, nbytes, (N,)))


def residual_norm_bwd(x: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor],
                      d_y: Optional[torch.Tensor], d_h: Optional[torch.Tensor] = None, *,
                      post_weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6,
                      workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None):
    """Backward of `residual_norm` (kda_residual_norm_bwd).  h as the forward returned it; d_y
    [T, N] in x's dtype (None exactly without `weight`) and d_h [T, N] in h's dtype (None: zero)
    are the gradients of y and h.  Returns (dx, d_residual in h's dtype, d_weight, d_post_weight,
    d_gate), None where the forward had no such argument (d_residual is always formed)."""
    if stream is not None:
        with _on(stream, x):
            return residual_norm_bwd(x, h, weight, d_y, d_h, post_weight=post_weight, gate=gate,
                                     scale=scale, eps=eps, workspace=workspace)
    scale, eps = float(scale), float(eps)
    key = ("residual_norm_bwd", _sig(x), _sig(h), _sig(weight), _sig(d_y), _sig(d_h),
           _sig(post_weight), _sig(gate), scale, eps)
    plan = _PLANS.get(key)
    if plan is None:
        plan = _plan_residual_norm_bwd(key, x, h, weight, d_y, d_h, post_weight, gate, scale, eps)
    dx = torch.empty_like(x)
    d_residual = torch.empty_like(h)
    d_weight = torch.empty_like(weight) if weight is not None else None
    d_post = torch.empty_like(post_weight) if post_weight is not None else None
    d_gate = None
    if gate is not None:
        d_gate = torch.empty(gate.shape, dtype=gate.dtype, device=plan.device)
    space, address, nbytes = _space(plan, workspace)
    _call(plan, x.data_ptr(), h.data_ptr(), _p(gate), _p(post_weight),
          _p(weight), _p(d_y), _p(d_h), dx.data_ptr(), d_residual.data_ptr(), _p(d_gate),
          _p(d_post), _p(d_weight), address, nbytes)
    return dx, d_residual, d_weight, d_post, d_gate


def _gated_params(o, gate, weight, y_dtype, activation, eps):
    if o.dim() != 3 or o.dtype not in _QKV_DTYPES or not o.is_contiguous():
        raise ValueError("o must be contiguous [T, H, D] float32 or bfloat16")
    T, H, D = o.shape
    if gate.shape != o.shape or gate.dtype not in _QKV_DTYPES:
        raise ValueError("gate must be [T, H, D] float32 or bfloat16")
    if activation not in _NORM_GATES:
        raise ValueError(f"activation must be one of {', '.join(_NORM_GATES)}")
    if y_dtype not in _QKV_DTYPES:
        raise ValueError("y must be float32 or bfloat16")
    _dense(weight, (D,), torch.float32, "weight")
    stride = 0
    if T > 0:
        if not gate[0].is_contiguous():
            raise ValueError("gate must have dense (H, D) rows")
        if T > 1:
            stride = gate.stride(0)
            if stride < H * D:
                raise ValueError("gate's rows must not overlap")
    return KdaNormParams(tokens=T, features=D, num_heads=H, x_dtype=_QKV_DTYPES[o.dtype],
                         gate_dtype=_QKV_DTYPES[gate.dtype], y_dtype=_QKV_DTYPES[y_dtype],
                         activation=_ACTIVATIONS[activation], eps=eps, scale=1.0,
                         gate_row_stride=stride)


def _plan_gated_norm(key, o, gate, weight, activation, eps, out_dtype, out):
    dev = _device(o, gate, weight, out)
    y_dtype = out.dtype if out is not None else (out_dtype or gate.dtype)
    p = _gated_params(o, gate, weight, y_dtype, activation, eps)
    if out is not None:
        _dense(out, o.shape, out_dtype or out.dtype, "out")
    return _keep(key, _Plan("kda_gated_norm_fwd", p, dev, 0, o.shape, y_dtype))


def gated_norm(o: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, *,
               activation: str = "sigmoid", eps: float = 1e-6,
               out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The output norm of the recurrence (kda_gated_norm_fwd): the RMS norm of each token's and
    head's o row, times weight [D], times act(gate).  o [T, H, D] as `prefill` and `decode_step`
    return it; gate [T, H, D] in either dtype, a column block of a packed projection if need be;
    `activation` of the gate: sigmoid, silu or none (the gate itself).  Returns y [T, H, D]
    (default the gate's dtype), ready as [T, H * D] for the output projection."""
    if stream is not None:
        with _on(stream, o):
            return gated_norm(o, gate, weight, activation=activation, eps=eps, out_dtype=out_dtype,
                              out=out)
    eps = float(eps)
    key = ("gated_norm", _sig(o), _sig(gate), _sig(weight), activation, eps, out_dtype, _sig(out))
    plan = _PLANS.get(key)
    if plan is None:
        plan = _plan_gated_norm(key, o, gate, weight, activation, eps, out_dtype, out)
    if out is None:
        out = torch.empty(plan.shape, dtype=plan.dtype, device=plan.device)
    _call(plan, o.data_ptr(), gate.data_ptr(), weight.data_ptr(),
          out.data_ptr())
    return out


def _plan_gated_norm_bwd(key, o, gate, weight, d_y, activation, eps):
    dev = _device(o, gate, weight, d_y)
    p = _gated_params(o, gate, weight, d_y.dtype, activation, eps)
    _dense(d_y, o.shape, d_y.dtype, "d_y")
    nbytes = _bytes("kda_norm_workspace_size", p, 1, dev)
    return _keep(key, _Plan("kda_gated_norm_bwd", p, dev, nbytes))


def gated_norm_bwd(o: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, d_y: torch.Tensor, *,
                   activation: str = "sigmoid", eps: float = 1e-6,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None):
    """Backward of `gated_norm` (kda_gated_norm_bwd).  Returns (d_o in o's dtype -- `prefill_bwd`'s
    d_o for the fp32 o of `prefill` --, d_gate dense in the gate's dtype, d_weight [D] float32)."""
    if stream is not None:
        with _on(stream, o):
            return gated_norm_bwd(o, gate, weight, d_y, activation=activation, eps=eps,
                                  workspace=workspace)
    eps = float(eps)
    key = ("gated_norm_bwd", _sig(o), _sig(gate), _sig(weight), _sig(d_y), activation, eps)
    plan = _PLANS.get(key)
    if plan is None:
        plan = _plan_gated_norm_bwd(key, o, gate, weight, d_y, activation, eps)
    d_o = torch.empty_like(o)
    d_gate = torch.empty(gate.shape, dtype=gate.dtype, device=plan.device)
    d_weight = torch.empty_like(weight)
    space, address, nbytes = _space(plan, workspace)
    _call(plan, o.data_ptr(), gate.data_ptr(), weight.data_ptr(),
          d_y.data_ptr(), d_o.data_ptr(), d_gate.data_ptr(), d_weight.data_ptr(), address, nbytes)
    return d_o, d_gate, d_weight
