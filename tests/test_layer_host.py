"""The layer's entry points without a GPU: every refusal comes back as a status before anything
touches CUDA, workspace sizes follow the parameters, and the binding refuses host tensors."""
import ctypes

import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib, build as kbuild, layer

P = ctypes.c_void_p
A = 1 << 20                       # an aligned address that is never read: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _lib.load()


def linear(**kw):
    base = dict(tokens=64, in_features=128, out_features=256, dtype=1, y_dtype=1, residual_dtype=1,
                dw_dtype=1, activation=0, scale=1.0)
    base.update(kw)
    return _lib.KdaLinearParams(**base)


def norm(**kw):
    base = dict(tokens=64, features=128, num_heads=4, x_dtype=1, h_dtype=1, gate_dtype=1, y_dtype=1,
                activation=_lib.KDA_ACT_SIGMOID, eps=1e-6, scale=1.0)
    base.update(kw)
    return _lib.KdaNormParams(**base)


def size(fn, p, flag):
    n = ctypes.c_size_t(0)
    return fn(ctypes.byref(p) if p is not None else None, flag, ctypes.byref(n)), n.value


def test_struct_layouts():
    assert ctypes.sizeof(_lib.KdaLinearParams) == 80
    assert _lib.KdaLinearParams.scale.offset == 36 and _lib.KdaLinearParams.x_row_stride.offset == 40
    assert ctypes.sizeof(_lib.KdaNormParams) == 56
    assert _lib.KdaNormParams.gate_row_stride.offset == 48


@pytest.mark.parametrize("kw,status", [
    (dict(), OK),
    (dict(tokens=0), OK),
    (dict(tokens=-1), INVALID),
    (dict(in_features=0), INVALID),
    (dict(out_features=0), INVALID),
    (dict(dtype=2), INVALID), (dict(y_dtype=-1), INVALID), (dict(residual_dtype=7), INVALID),
    (dict(dw_dtype=2), INVALID),
    (dict(activation=5), INVALID), (dict(activation=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(flags=1), INVALID), (dict(flags=4), INVALID), (dict(flags=128), INVALID),
    (dict(flags=_lib.KDA_FLAG_CUDA_CORES | _lib.KDA_FLAG_UNALIGNED_X), OK),
    (dict(x_row_stride=127), INVALID), (dict(w_row_stride=-128), INVALID),
    (dict(y_row_stride=255), INVALID), (dict(residual_row_stride=1), INVALID),
    (dict(x_row_stride=1 << 50), INVALID),
    (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(in_features=(1 << 24) + 1), UNSUPPORTED),
])
@pytest.mark.parametrize("backward", [0, 1])
def test_linear_params(lib, kw, status, backward):
    assert size(lib.kda_linear_workspace_size, linear(**kw), backward)[0] == status


def test_linear_workspace(lib):
    def fwd(**kw):
        return size(lib.kda_linear_workspace_size, linear(**kw), 0)[1]

    def bwd(**kw):
        return size(lib.kda_linear_workspace_size, linear(**kw), 1)[1]
    assert fwd() == 0                                     # aligned bf16 rows are read in place
    assert fwd(x_row_stride=129) >= 64 * 128 * 2          # a copy of x
    assert fwd(w_row_stride=130) >= 256 * 128 * 2
    assert fwd(flags=_lib.KDA_FLAG_UNALIGNED_W) >= 256 * 128 * 2
    assert fwd(dtype=0, y_dtype=0) >= (64 + 256) * 128 * 6       # three bf16 planes of each
    assert fwd(dtype=0, y_dtype=0, flags=_lib.KDA_FLAG_CUDA_CORES) == 0
    assert fwd(dtype=0, y_dtype=0, tokens=8) == 0         # few tokens: read in place
    assert bwd(activation=2) >= bwd() + 64 * 256 * 2      # dz
    assert bwd(y_dtype=0) >= bwd() + 64 * 256 * 2
    assert size(lib.kda_linear_workspace_size, None, 0)[0] == INVALID
    assert lib.kda_linear_workspace_size(ctypes.byref(linear()), 0, None) == INVALID


def test_linear_pointers(lib):
    def fwd(p=None, x=A, w=A, b=None, r=None, y=A, z=None, ws=None, n=0):
        return lib.kda_linear_fwd(ctypes.byref(p or linear()), x, w, b, r, y, z, ws, n, None)
    assert lib.kda_linear_fwd(None, A, A, None, None, A, None, None, 0, None) == INVALID
    assert fwd(p=linear(tokens=0), x=None, w=None, y=None) == OK        # nothing to do
    assert fwd(x=None) == INVALID and fwd(w=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(x=A + 1) == INVALID and fwd(y=A + 1) == INVALID and fwd(b=A + 2) == INVALID
    assert fwd(r=A + 1) == INVALID and fwd(z=A + 1) == INVALID
    assert fwd(x=A + 2) == INVALID                        # unaligned base without its flag
    p = linear(flags=_lib.KDA_FLAG_UNALIGNED_X)
    assert fwd(p=p, x=A + 2) == WORKSPACE                 # announced: a copy, so a workspace
    need = size(lib.kda_linear_workspace_size, p, 0)[1]
    assert fwd(p=p, x=A + 2, ws=A, n=need - 1) == WORKSPACE
    assert fwd(p=p, x=A + 2, ws=A + 16, n=need) == WORKSPACE   # not 256-byte aligned

    def bwd(p=None, x=A, w=A, z=None, dy=A, dx=A, dw=A, db=None, ws=A, n=1 << 40):
        return lib.kda_linear_bwd(ctypes.byref(p or linear()), x, w, z, dy, dx, dw, db, ws, n, None)
    assert bwd(dy=None) == INVALID and bwd(w=None) == INVALID and bwd(x=None) == INVALID
    assert bwd(p=linear(activation=2)) == INVALID         # needs the pre-activation
    assert bwd(dx=A + 1) == INVALID and bwd(db=A + 2) == INVALID and bwd(dy=A + 2) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(n=0) == WORKSPACE


@pytest.mark.parametrize("kw,gated,status", [
    (dict(), 0, OK), (dict(), 1, OK), (dict(tokens=0), 0, OK), (dict(tokens=0), 1, OK),
    (dict(tokens=-1), 0, INVALID), (dict(features=0), 1, INVALID), (dict(num_heads=0), 1, INVALID),
    (dict(x_dtype=3), 0, INVALID), (dict(h_dtype=3), 0, INVALID), (dict(gate_dtype=3), 1, INVALID),
    (dict(y_dtype=0), 0, INVALID),                        # y has x's dtype
    (dict(y_dtype=0), 1, OK),
    (dict(eps=0.0), 0, INVALID), (dict(eps=-1.0), 1, INVALID), (dict(eps=float("nan")), 0, INVALID),
    (dict(scale=float("inf")), 0, INVALID),
    (dict(activation=_lib.KDA_ACT_GELU), 1, INVALID), (dict(activation=_lib.KDA_ACT_RELU), 1, INVALID),
    (dict(gate_row_stride=127), 0, INVALID), (dict(gate_row_stride=511), 1, INVALID),
    (dict(features=16385), 0, UNSUPPORTED), (dict(features=1025), 1, UNSUPPORTED),
    (dict(tokens=1 << 31), 0, UNSUPPORTED), (dict(tokens=1 << 30), 1, UNSUPPORTED),
])
def test_norm_params(lib, kw, gated, status):
    assert size(lib.kda_norm_workspace_size, norm(**kw), gated)[0] == status


def test_norm_pointers(lib):
    def fwd(p=None, x=A, r=None, g=None, pw=None, w=A, h=A, y=A):
        return lib.kda_residual_norm_fwd(ctypes.byref(p or norm()), x, r, g, pw, w, h, y, None)
    assert fwd(p=norm(tokens=0), x=None, y=None) == OK
    assert fwd(x=None) == INVALID and fwd(w=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(w=None, y=None, h=None) == INVALID         # nothing to write
    assert fwd(x=A + 1) == INVALID and fwd(w=A + 2) == INVALID and fwd(g=A + 2) == INVALID
    assert fwd(p=norm(gate_per_token=1), g=A + 1) == INVALID

    def bwd(p=None, x=A, h=A, g=None, pw=None, w=A, dy=A, dh=None, dx=A, dr=A, dg=None, dpw=None,
            dw=A, ws=A, n=1 << 40):
        return lib.kda_residual_norm_bwd(ctypes.byref(p or norm()), x, h, g, pw, w, dy, dh, dx, dr,
                                         dg, dpw, dw, ws, n, None)
    assert bwd(dy=None) == INVALID                        # comes with weight
    assert bwd(w=None, dy=None, dw=None) == INVALID       # no gradient at all
    assert bwd(dx=None) == INVALID and bwd(h=None) == INVALID and bwd(dw=None) == INVALID
    assert bwd(g=A) == INVALID and bwd(pw=A) == INVALID   # their gradients are missing
    assert bwd(g=A, dg=A, x=None) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(n=16) == WORKSPACE

    def gf(p=None, o=A, g=A, w=A, y=A):
        return lib.kda_gated_norm_fwd(ctypes.byref(p or norm()), o, g, w, y, None)
    assert gf(p=norm(tokens=0), o=None, g=None, y=None) == OK
    assert gf(o=None) == INVALID and gf(g=None) == INVALID and gf(w=None) == INVALID
    assert gf(y=None) == INVALID and gf(g=A + 1) == INVALID

    def gb(p=None, o=A, g=A, w=A, dy=A, do=A, dg=A, dw=A, ws=A, n=1 << 40):
        return lib.kda_gated_norm_bwd(ctypes.byref(p or norm()), o, g, w, dy, do, dg, dw, ws, n, None)
    assert gb(dy=None) == INVALID and gb(do=None) == INVALID and gb(dw=None) == INVALID
    assert gb(ws=A + 8) == WORKSPACE and gb(n=0) == WORKSPACE


def test_binding_refuses_host_tensors_and_bad_shapes():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    v = torch.zeros(8)
    o = torch.zeros(2, 3, 8)
    for call in (lambda: kda.linear(x, w), lambda: kda.linear_bwd(x, w, torch.zeros(4, 6)),
                 lambda: kda.residual_norm(x, v), lambda: kda.residual_norm_bwd(x, x, v, x),
                 lambda: kda.gated_norm(o, o, v), lambda: kda.gated_norm_bwd(o, o, v, o)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("call", [
    lambda x, w: layer._linear_params(x[0], w, "none", 1.0, x.dtype, 0),        # not [T, K]
    lambda x, w: layer._linear_params(x, w[:, :7], "none", 1.0, x.dtype, 0),    # another K
    lambda x, w: layer._linear_params(x, w.bfloat16(), "none", 1.0, x.dtype, 0),
    lambda x, w: layer._linear_params(x.half(), w.half(), "none", 1.0, x.dtype, 0),
    lambda x, w: layer._linear_params(x, w, "tanh", 1.0, x.dtype, 0),
    lambda x, w: layer._linear_params(x, w, "none", 1.0, torch.float16, 0),
    lambda x, w: layer._linear_params(x.t().contiguous().t(), w, "none", 1.0, x.dtype, 0),
    lambda x, w: layer._linear_params(x[:1].expand(4, 8), w, "none", 1.0, x.dtype, 0),
    lambda x, w: layer._residual_params(x[:, ::2], x.dtype, 1.0, 1e-6),
    lambda x, w: layer._gated_params(x.view(2, 2, 8), x.view(2, 2, 8), w[0, :7], x.dtype, "silu", 1e-6),
    lambda x, w: layer._gated_params(x.view(2, 2, 8), x.view(2, 2, 8), w[0], x.dtype, "gelu", 1e-6),
    lambda x, w: layer._gated_params(x.view(2, 2, 8), x.view(2, 2, 8)[:1].expand(2, 2, 8), w[0],
                                     x.dtype, "silu", 1e-6),
])
def test_binding_checks(call):
    with pytest.raises(ValueError):
        call(torch.zeros(4, 8), torch.zeros(6, 8))
