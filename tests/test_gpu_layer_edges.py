"""Calls of the layer's operators at the edges of their range that `test_gpu_layer.py` does not make:
shares of a split sum, tile widths, tails of the activations, infinities, calls from several
threads.  Tolerances as there.
"""
import ctypes
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib, build as kbuild
from oracle import layer as ol
from test_gpu_layer import DEV, U, check, dev, host, linear_case, no_error, product_tol, rng

pytestmark = pytest.mark.gpu
erfc64 = np.vectorize(math.erfc, otypes=[np.float64])


@pytest.mark.parametrize("T", [3, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("K,N", [(4096, 512), (1024, 256)])
@pytest.mark.parametrize("dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_split_sums_of_few_rows_back_to_back(T, K, N, dtype, y):
    """Few rows give only some CTAs of a cluster columns to finish, and the others end once their
    shares have arrived.  Launched back to back with kernels that take over their shared memory
    at once, every call gives the same bits, and the fp64 sum."""
    r = rng(30, T, K)
    x, x64 = dev(r.standard_normal((T, K)), dtype)
    w, w64 = dev(r.standard_normal((N, K)) / np.sqrt(K), dtype)
    other, _ = dev(r.standard_normal((T + 5, K)), dtype)
    yt = torch.float32 if y == "f32" else torch.bfloat16
    outs = []
    for _ in range(40):
        outs.append(kda.linear(x, w, out_dtype=yt))
        kda.linear(other, w, out_dtype=yt)
    no_error()
    check("y", outs[0], x64 @ w64.T, product_tol(x64, w64.T, K, dtype))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.fixture(scope="module")
def giving_up(tmp_path_factory):
    """The row kernels with waits that give up at once."""
    lib = str(tmp_path_factory.mktemp("ring") / "libring.so")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, *kbuild.NVCC_FLAGS, "-DKDA_ROW_WAIT=0", "-shared", "-o", lib,
                    os.path.join(os.path.dirname(__file__), "ring_gives_up.cu")], check=True)
    f = ctypes.CDLL(lib).ring_gives_up
    f.argtypes = [ctypes.POINTER(_lib.KdaNormParams), ctypes.c_int] + [ctypes.c_void_p] * 10
    return f


@pytest.mark.parametrize("T,N,backward", [(15000, 96, 0), (15000, 96, 1), (5000, 2048, 0), (5000, 2048, 1),
                                          (3000, 4096, 0), (3000, 4096, 1), (1000, 16384, 1)])
def test_rows_whose_wait_gives_up_end_with_their_copies(giving_up, T, N, backward):
    """A wait that gives up is an error in the device word; the block ends only after the copies it
    asked for, so that a kernel behind it finds its own shared memory untouched."""
    r = rng(31, T, N)
    x, _ = dev(r.standard_normal((T, N)), "bf16")
    w, _ = dev(r.standard_normal(N), "f32")
    want = kda.residual_norm(x, w, residual=x) + kda.residual_norm_bwd(x, x, w, x, x)[:3]
    p = _lib.KdaNormParams(tokens=T, features=N, x_dtype=1, h_dtype=1, y_dtype=1, eps=1e-6, scale=1.0)
    n = ctypes.c_size_t(0)
    assert _lib.load().kda_norm_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device=DEV)
    dx, dh, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(5):
        assert giving_up(ctypes.byref(p), backward, x.data_ptr(), x.data_ptr(), w.data_ptr(), x.data_ptr(),
                         dx.data_ptr(), dh.data_ptr(), dw.data_ptr(), ws.data_ptr(), word.data_ptr(),
                         torch.cuda.current_stream().cuda_stream) == 0
        got = kda.residual_norm(x, w, residual=x) + kda.residual_norm_bwd(x, x, w, x, x)[:3]
        no_error()
        assert word.item() == _lib.KDA_DEVERR_TIMEOUT
        for a, b in zip(got, want):
            assert torch.equal(a, b)


class ThreadArgs(ctypes.Structure):
    """Mirror of Args in call_from_threads.cpp."""

    _fields_ = ([("p", ctypes.POINTER(_lib.KdaNormParams))] + [(n, ctypes.c_void_p) for n in (
        "x", "h", "gate", "post_weight", "weight", "d_y", "d_h", "dx", "d_residual", "d_gate",
        "d_post_weight", "d_weight", "workspace")] + [("workspace_bytes", ctypes.c_size_t),
                                                      ("stream", ctypes.c_void_p)])


def test_two_widths_from_two_threads(tmp_path):
    """Host threads that call one kernel with rings of different sizes (2048 columns: 40 KB, 4096: 80
    KB) do not disturb each other."""
    so = str(tmp_path / "libthreads.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I", kbuild.INCLUDE, "-o", so,
                    os.path.join(os.path.dirname(__file__), "call_from_threads.cpp")], check=True)
    run = ctypes.CDLL(so).call_from_threads
    lib = _lib.load()
    args, want, got, keep = (ThreadArgs * 4)(), [], [], []
    for i in range(4):
        T, N = 2500, (2048, 4096)[i % 2]
        r = rng(32, i)
        x, _ = dev(r.standard_normal((T, N)), "bf16")
        g, _ = dev(r.standard_normal((T, N)), "bf16")
        w, _ = dev(r.standard_normal(N), "f32")
        want.append(kda.residual_norm_bwd(x, x, w, x, x, post_weight=w, gate=g))
        p = _lib.KdaNormParams(tokens=T, features=N, x_dtype=1, h_dtype=1, y_dtype=1, gate_per_token=1, eps=1e-6,
                               scale=1.0)
        n = ctypes.c_size_t(0)
        assert lib.kda_norm_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == 0
        ws = torch.empty(n.value, dtype=torch.uint8, device=DEV)
        out = [torch.empty_like(t) for t in want[-1]]
        s = torch.cuda.Stream()
        a, c, e = x.data_ptr(), w.data_ptr(), [t.data_ptr() for t in out]
        args[i] = ThreadArgs(ctypes.pointer(p), a, a, g.data_ptr(), c, c, a, a, e[0], e[1], e[4], e[3], e[2],
                             ws.data_ptr(), n.value, s.cuda_stream)
        got.append(out)
        keep.append((p, x, g, w, ws, s))
    torch.cuda.synchronize()
    assert run(ctypes.cast(lib.kda_residual_norm_bwd, ctypes.c_void_p), args, 4, 2000) == 0
    no_error()
    for a, b in zip(got, want):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T", [65, 100, 128])
@pytest.mark.parametrize("dtype,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_few_tokens_onto_more_rows_than_one_wave(T, dtype, y):
    """A vocabulary-sized weight: more 128-row tiles than SMs."""
    N = 128 * torch.cuda.get_device_properties(0).multi_processor_count + 136
    linear_case(33, T, 136, N, dtype, act="silu", bias=True, res=y, y=y, scale=0.5)


# ------------------------------------------------------- tile widths of the persistent product

WIDTHS = (256, 224, 192, 160, 128)


def width_rule():
    """The widths and their costs as the library's source states them."""
    src = open(os.path.join(kbuild.CSRC, "linear_tc.cuh")).read()
    w, c = re.search(r"kWidth\[5\] = \{([\d, ]+)\}, kCost\[5\] = \{([\d, ]+)\}", src).groups()
    return [int(v) for v in w.split(",")], [int(v) for v in c.split(",")]


def shape_of_width(want):
    """Output columns and rows (I, J), odd in both tiles, for which the library takes tiles `want` wide:
    at least two whole ones and a ragged one along J."""
    widths, costs = width_rule()
    assert tuple(widths) == WIDTHS
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    best = None
    for ti in range(2, 24):
        I = 256 * ti - 104
        for J in range(2 * want + 10, 4000, 14):
            if ti * -(-J // 256) < sms // 4 or best and I * J >= best[0] * best[1]:
                continue
            waves = [-(-ti * -(-J // w) // (sms // 2)) * c for w, c in zip(widths, costs)]
            if widths[waves.index(min(waves))] == want:
                best = I, J
    assert best, want
    return best


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("form", ["plain", "z", "in place", "fp32 residual", "fp32"])
def test_forward_at_each_tile_width(width, form):
    N, T = shape_of_width(width)
    K = 200
    r = rng(34, width)
    x, x64 = dev(r.standard_normal((T, K)), "bf16")
    w, w64 = dev(r.standard_normal((N, K)) / np.sqrt(K), "bf16")
    b, b64 = dev(r.standard_normal(N), "f32")
    kw = dict(activation="silu", scale=0.5, out_dtype=torch.float32 if form == "fp32" else torch.bfloat16)
    rs, rs64, z = None, None, None
    if form in ("in place", "fp32 residual"):
        rs, rs64 = dev(r.standard_normal((T, N)), "bf16" if form == "in place" else "f32")
    if form in ("z", "fp32 residual"):
        y, z = kda.linear(x, w, b, residual=rs, save_pre_activation=True, **kw)
    else:
        y = kda.linear(x, w, b, residual=rs, out=rs if form == "in place" else None, **kw)
    no_error()
    y_ref, z_ref = ol.linear(x64, w64, b64, "silu", rs64, 0.5)
    ez = product_tol(x64, w64.T, K, "bf16") + 2 * U * np.abs(z_ref)
    check("y", y, y_ref, 0.5 * (1.13 * ez + 16 * U * np.maximum(1, np.abs(z_ref))) + 4 * U * np.abs(y_ref))
    if z is not None:
        check("z", z, z_ref, ez)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dw_dtype", ["bf16", "f32"])
def test_gradients_at_each_tile_width(width, dw_dtype):
    I, J = shape_of_width(width)
    C = 328
    r = rng(35, width)
    # dx [T = J, K = I], summed over N = C
    w, w64 = dev(r.standard_normal((C, I)), "bf16")
    d, d64 = dev(r.standard_normal((J, C)), "bf16")
    x, _ = dev(r.standard_normal((J, I)), "bf16")
    dx = kda.linear_bwd(x, w, d, need_dw=False, scale=-1.5)[0]
    no_error()
    ref = -1.5 * (d64 @ w64)
    check("dx", dx, ref, 1.5 * product_tol(d64, w64, C, "bf16") + 2 * U * np.abs(ref))
    # dw [N = J, K = I], summed over T = C
    x, x64 = w, w64
    d, d64 = dev(r.standard_normal((C, J)), "bf16")
    w, _ = dev(r.standard_normal((J, I)), "bf16")
    dw = kda.linear_bwd(x, w, d, need_dx=False, dw_dtype=torch.float32 if dw_dtype == "f32" else torch.bfloat16)[1]
    no_error()
    ref = d64.T @ x64
    check("dw", dw, ref, product_tol(d64.T, x64, C, "bf16") + 2 * U * np.abs(ref))


@pytest.mark.parametrize("K", [64, 200, 700])
def test_pair_products_back_to_back(K):
    """The pair's last releases arrive in both CTAs' shared memory: launched back to back with kernels
    that take it over at once, among them short sums that end right behind their last products, every
    call gives the same bits."""
    r = rng(37, K)
    x, x64 = dev(r.standard_normal((1664, K)), "bf16")
    w, w64 = dev(r.standard_normal((1600, K)), "bf16")
    few = x[:40].contiguous()
    v = torch.ones(1600, device=DEV)
    outs = []
    for _ in range(40):
        outs.append(kda.linear(x, w))
        kda.linear(few, w)
        kda.residual_norm(outs[-1], v, residual=outs[-1])
    no_error()
    check("y", outs[0], x64 @ w64.T, product_tol(x64, w64.T, K, "bf16"))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


# ------------------------------------------------------------------- the far side of the activations

@pytest.mark.parametrize("act", ["gelu", "silu", "sigmoid"])
@pytest.mark.parametrize("T", [1, 9, 600])
def test_activation_tails_keep_their_relative_size(act, T):
    """Far below zero gelu, silu and sigmoid are tiny and still right to their type's rounding: half a
    bf16 step, plus 2e-4 (the normal distribution's approximation 1e-4; exp of an argument a up to 78
    that is itself rounded, (2 + 1.2 a) 2^-23 + 4 a 2^-24 < 3e-5).  One row, few rows and many take
    three kernels."""
    N, K = 4096, 64
    z = np.linspace(-12.5, 9, N).astype(np.float32)
    b = torch.from_numpy(z).to(DEV)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    y = kda.linear(x, w, b, activation=act)
    no_error()
    ref = z * 0.5 * erfc64(-z / math.sqrt(2)) if act == "gelu" else ol.act(act, z)
    check("y", y, np.broadcast_to(ref, (T, N)), 2e-4 * np.abs(ref))


@pytest.mark.parametrize("act", ["gelu", "silu", "sigmoid"])
def test_activation_gradient_tails_keep_their_relative_size(act):
    """The same of the slopes of a bf16 pre-activation below -2, where no two terms cancel but gelu's
    two (each within 2e-4, the smaller at most a fifth of the difference)."""
    N, K = 1024, 64
    z = torch.linspace(-12.5, -2, N, device=DEV).to(torch.bfloat16)[None]
    x = torch.zeros((1, K), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    db = kda.linear_bwd(x, w, torch.ones_like(z), activation=act, pre_activation=z, need_dx=False, need_dw=False,
                        need_bias=True)[2]
    no_error()
    z64 = host(z)[0]
    ref = (0.5 * erfc64(-z64 / math.sqrt(2)) + z64 * np.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
           if act == "gelu" else ol.act_grad(act, z64))
    check("db", db, ref, 3e-4 * np.abs(ref))


# ------------------------------------------------------------------- infinities in fp32 operands

def same(got, ref):
    """Equal in every infinity's sign and place, and in the places of NaN."""
    g, r = got.cpu(), ref.cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(r))
    assert torch.equal(torch.isposinf(g), torch.isposinf(r)) and torch.equal(torch.isneginf(g), torch.isneginf(r))


@pytest.mark.parametrize("T", [1, 8, 9, 64, 150, 700])
@pytest.mark.parametrize("K,N", [(64, 72), (1100, 200)])
def test_fp32_infinities_stay_infinities(T, K, N):
    """An infinite or NaN term gives what fp32 sums give, for every row count: its infinity, or NaN
    next to a zero, to another sign's infinity or to NaN."""
    r = rng(36, T, K)
    x = torch.from_numpy(r.standard_normal((T, K)).astype(np.float32))
    w = torch.from_numpy(r.standard_normal((N, K)).astype(np.float32))
    x[0, 5] = float("inf")
    w[3, 5] = 0
    w[7, K - 1] = float("-inf")
    if T > 5:
        x[2, 9] = float("nan")
        x[4, 1], x[4, K - 2] = float("inf"), float("-inf")
        x[5, K - 1] = float("-inf")
    d = torch.from_numpy(r.standard_normal((T, N)).astype(np.float32))
    if T > 5:
        d[1, 11] = float("inf")
    xg, wg, dg = x.to(DEV), w.to(DEV), d.to(DEV)
    y = kda.linear(xg, wg)
    dx, dw, db = kda.linear_bwd(xg, wg, dg, need_bias=True)
    no_error()
    same(y, x.double() @ w.double().t())
    same(dx, d.double() @ w.double())
    same(dw, d.double().t() @ x.double())
    same(db, d.double().sum(0))
    clean = [t for t in range(T) if t not in (0, 2, 4, 5)]
    other = [n for n in range(N) if n != 7]
    if clean:
        x64, w64 = x.double().numpy()[clean], w.double().numpy()[other]
        check("y", y[clean][:, other], x64 @ w64.T, product_tol(x64, w64.T, K, "f32"))


def test_fp32_products_next_to_the_largest_value():
    """Terms just below fp32's largest value stay finite: their leading parts round up past it."""
    T, K, N = 40, 64, 48
    x = torch.zeros((T, K), device=DEV)
    w = torch.zeros((N, K), device=DEV)
    a = 2.0 ** 64 * (1 - 2.0 ** -24)                         # its square lies a step below the largest value
    x[:, 3], w[:, 3] = a, a
    x[:, 7], w[:, 7] = 1.0, -(2.0 ** 100)
    y = kda.linear(x, w)
    no_error()
    ref = np.full((T, N), a * a - 2.0 ** 100)
    check("y", y, ref, 4 * U * ref)


FIRST_CALLS = """
import torch, gated_delta_rule_deltanet_gb300 as kda
r = torch.Generator(device="cuda").manual_seed(1)
x, w, d = (torch.randn(s, generator=r, device="cuda").bfloat16() for s in ((64, 256), (512, 256), (64, 512)))
v, o = torch.randn(256, generator=r, device="cuda"), torch.randn((64, 2, 128), generator=r, device="cuda")
def calls():
    out = [kda.linear(x, w)] + list(kda.linear_bwd(x, w, d, need_bias=True))
    out += [*kda.residual_norm(x, v, residual=x), *kda.residual_norm_bwd(x, x, v, x)[:3]]
    return out + [kda.gated_norm(o, o, v[:128]), *kda.gated_norm_bwd(o, o, v[:128], o)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = calls()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, calls())) and kda.get_device_error() == 0
"""


def test_first_calls_of_a_process_may_be_captured():
    """What the library sets up on its first calls (limits, the error word, maps) is allowed in a
    capture."""
    subprocess.run([sys.executable, "-c", FIRST_CALLS], check=True, cwd=kbuild.ROOT, timeout=300)
