"""The layer around the recurrence (linear, residual_norm, gated_norm and their gradients) on the
GPU against the fp64 reference of `oracle/layer.py`.

Tolerances, element by element, from the arithmetic (U = 2^-24 is fp32's rounding, R(t) half a
step of the stored type, `torch.finfo(t).eps / 2` relative to the value):

  sums of K products  the products of two bf16 are exact in fp32; each of the K additions is off
                      by at most one unit in the last place of a partial sum, 2 U sum|a b| (the
                      tensor cores may truncate); fp32 products add U each
  row norms           the mean square adds N terms of one sign in chains of at most 40 (eight to
                      32 elements a thread, then a tree): 40 U relative, half of it in the root;
                      with the element's own few products 64 U covers each factor
  column sums         T additions: (T + 64) U sum|terms|
  activations         within 16 U of a value of size max(1, |z|); slope at most 1.13
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
import oracle
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def R(t):
    return torch.finfo(t).eps / 2


def rng(*seed):
    return np.random.Generator(np.random.PCG64([*seed]))


def dev(a, dtype):
    """The array on the GPU in `dtype`, and the values it then holds in fp64."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype])
    return t.to(DEV), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def check(name, got, ref, tol):
    """|got - ref| <= tol plus the rounding of the stored type."""
    g = host(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if g.size == 0:
        return
    assert np.all(np.isfinite(g)), f"{name}: non-finite"
    lim = np.broadcast_to(tol, ref.shape)
    lim = lim + R(got.dtype) * (np.abs(ref) + lim) + 1e-37
    bad = np.abs(g - ref) > lim
    i = np.unravel_index(np.argmax(np.abs(g - ref) / lim), ref.shape)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst at {i}: {g[i]} for {ref[i]}, limit {lim[i]}"


def no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


# ------------------------------------------------------------------------------------------ linear

def product_tol(a, b, C, dtype):
    return (2 * C + (0 if dtype == "bf16" else 1)) * U * (np.abs(a) @ np.abs(b))


def linear_case(seed, T, K, N, dtype, *, act="none", bias=False, res=None, scale=1.0, y=None,
                cuda_cores=False, views=lambda t: t):
    """Runs forward and backward and checks every output."""
    r = rng(seed, T, K, N)
    x, x64 = dev(r.standard_normal((T, K)), dtype)
    w, w64 = dev(r.standard_normal((N, K)) / np.sqrt(K), dtype)
    x, w = views(x), views(w)
    b, b64 = dev(r.standard_normal(N) * 0.3, "f32") if bias else (None, None)
    rs, rs64 = dev(r.standard_normal((T, N)), res) if res else (None, None)
    yt = DT[y or dtype]
    out, z = kda.linear(x, w, b, activation=act, residual=views(rs) if res else None, scale=scale,
                        out_dtype=yt, save_pre_activation=True, cuda_cores=cuda_cores)
    plain = kda.linear(x, w, b, activation=act, residual=rs, scale=scale, out_dtype=yt,
                       cuda_cores=cuda_cores)
    no_error()
    assert out.dtype == yt and z.dtype == DT[dtype]
    assert torch.equal(plain, out)
    y_ref, z_ref = ol.linear(x64, w64, b64, act, rs64, scale)
    ez = product_tol(x64, w64.T, K, dtype) + 2 * U * np.abs(z_ref)
    check("z", z, z_ref, ez)
    ey = abs(scale) * (1.13 * ez + 16 * U * np.maximum(1, np.abs(z_ref))) + 4 * U * np.abs(y_ref)
    check("y", out, y_ref, ey)

    dy, dy64 = dev(r.standard_normal((T, N)) * 1e-2, y or dtype)
    z64 = host(z)
    dx, dw, db = kda.linear_bwd(x, w, views(dy), activation=act, pre_activation=z, scale=scale,
                                need_bias=True, cuda_cores=cuda_cores)
    dw32 = kda.linear_bwd(x, w, dy, activation=act, pre_activation=z, scale=scale, need_dx=False,
                          dw_dtype=torch.float32, cuda_cores=cuda_cores)[1]
    no_error()
    dx_ref, dw_ref, db_ref, dz = ol.linear_bwd(x64, w64, dy64, z64, act, scale)
    az = np.abs(dz)
    # slopes within 32 U of a value below 1.13; rounded to the operand type where it is formed
    formed = act != "none" or (y or dtype) != dtype
    ed = (32 * U + (R(DT[dtype]) if formed else 0)) * np.maximum(az, abs(scale) * np.abs(dy64) * (act != "none"))
    check("dx", dx, dx_ref, product_tol(dz, w64, N, dtype) + ed @ np.abs(w64) + 2 * U * np.abs(dx_ref))
    ew = product_tol(dz.T, x64, T, dtype) + ed.T @ np.abs(x64) + 2 * U * np.abs(dw_ref)
    check("dw", dw, dw_ref, ew)
    check("dw32", dw32, dw_ref, ew)
    check("db", db, db_ref, (T + 64) * U * az.sum(0) + 32 * U * (abs(scale) * np.abs(dy64)).sum(0))


SHAPES = [(1, 64, 16), (1, 1, 1), (3, 7, 5), (17, 100, 33), (64, 128, 128), (129, 256, 257),
          (200, 520, 130), (256, 64, 384), (300, 72, 24), (1, 2048, 640), (33, 1000, 264)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_shapes(T, K, N, dtype):
    linear_case(1, T, K, N, dtype, bias=True)


@pytest.mark.parametrize("dtype,y,res,K", [("bf16", "bf16", "f32", 200), ("bf16", "f32", "f32", 1100),
                                           ("bf16", "f32", "bf16", 1100), ("bf16", "f32", None, 1100)])
def test_linear_pair_tiles_of_other_types(dtype, y, res, K):
    """Residuals that are and are not of y's type, and fp32 results, at the persistent kernel's
    sizes (its backward then has an fp32 d_y)."""
    linear_case(12, 1601, K, 1608, dtype, act="sigmoid", bias=True, res=res, y=y, scale=-1.5)


def test_linear_pair_tiles_in_place():
    r = rng(13)
    T, K, N = 1700, 128, 1600
    x, x64 = dev(r.standard_normal((T, K)), "bf16")
    w, w64 = dev(r.standard_normal((N, K)), "bf16")
    for dtype in ("bf16", "f32"):
        h, h64 = dev(r.standard_normal((T, N)), dtype)
        y = kda.linear(x, w, residual=h, out=h, scale=0.5)
        no_error()
        assert y is h
        ref = ol.linear(x64, w64, None, "none", h64, 0.5)[0]
        check("y", h, ref, product_tol(x64, w64.T, K, "bf16") + 4 * U * np.abs(ref))


def test_arrays_past_2_to_the_31():
    """More than 2^31 elements: the last rows equal those of a call on the last rows alone."""
    T, N = 530000, 4160                                    # 2.2e9 elements
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn((T, 64), generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn((N, 64), generator=g, device=DEV, dtype=torch.bfloat16)
    y = kda.linear(x, w)
    tail = slice(T - 300, T)
    assert torch.equal(y[tail], kda.linear(x[tail].contiguous(), w))
    dx = kda.linear_bwd(x, w, y, need_dw=False)[0]
    ref = y[tail].float() @ w.float()
    assert (dx[tail].float() - ref).abs().max() <= 2 * R(torch.bfloat16) * ref.abs().max()
    del dx
    v = torch.randn(N, generator=g, device=DEV)
    n, h = kda.residual_norm(y, v, residual=y)
    yt = y[tail].contiguous()
    nt, ht = kda.residual_norm(yt, v, residual=yt)
    # another kernel (rows read directly): the order of a row's sum may differ, a bf16 step then
    assert torch.equal(h[tail], ht) and (n[tail].float() - nt.float()).abs().max() <= 2 * R(torch.bfloat16) * nt.abs().max()
    del n, h
    o = y.view(-1)[:T * N // 128 * 128].view(-1, 1, 128)
    z = kda.gated_norm(o, o, v[:128].contiguous())
    zt = kda.gated_norm(o[-500:].contiguous(), o[-500:].contiguous(), v[:128].contiguous())
    no_error()
    assert torch.equal(z[-500:], zt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(64, 4096, 64), (1500, 2112, 1600), (300, 1100, 200)])
def test_linear_fp32_results_round_like_fp32_sums(T, K, N, dtype):
    """A long sum with an fp32 result is not left to the truncating accumulators: relative to the
    result's norm it stays within sqrt(K) roundings (an fp32 chain's random walk), 2 of them
    for the systematic part."""
    r = rng(11, T, K)
    x, x64 = dev(r.standard_normal((T, K)), dtype)
    w, w64 = dev(r.standard_normal((N, K)) / np.sqrt(K), dtype)
    d, d64 = dev(r.standard_normal((T, N)), dtype)
    y = host(kda.linear(x, w, out_dtype=torch.float32))
    dw = host(kda.linear_bwd(x, w, d, need_dx=False, dw_dtype=torch.float32)[1])
    no_error()
    for got, ref, c in ((y, x64 @ w64.T, K), (dw, d64.T @ x64, T)):
        # up to 1024 steps stay in one accumulator: 64 truncations of up to 2 U each, half on average
        lim = 2 * np.sqrt(c) * U if c > 1024 else max(2 * np.sqrt(c), c / 16) * U
        assert np.linalg.norm(got - ref) <= lim * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("K,N", [(520, 70), (4096, 40), (37, 261)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_few_tokens(T, K, N, dtype):
    linear_case(10, T, K, N, dtype, act="silu", bias=True, res=dtype, scale=0.5)


@pytest.mark.parametrize("T,K,N", [(1664, 1600, 1664), (1700, 1540, 1603)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_pair_tiles(T, K, N, dtype):
    """Products of enough 256 x 256 tiles for the persistent kernel, with ragged edges."""
    linear_case(9, T, K, N, dtype, act="silu", bias=True, res=dtype)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dtype,y,res", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                         ("f32", "f32", "f32"), ("f32", "bf16", "bf16"),
                                         ("bf16", "bf16", "f32")])
def test_linear_epilogue(act, dtype, y, res):
    linear_case(2, 77, 192, 136, dtype, act=act, bias=True, res=res, scale=0.5, y=y)


def test_linear_cuda_cores_path():
    linear_case(3, 140, 96, 150, "bf16", act="silu", bias=True, cuda_cores=True)


@pytest.mark.parametrize("K", [1, 3, 66, 2047, 2049, 4161])
@pytest.mark.parametrize("off", [0, 1, 2, 5])
def test_linear_copies_of_unaligned_rows(K, off):
    """Widths around the copy's word and stretch sizes, from even and odd elements."""
    r = rng(14, K, off)
    T, N = 20, 24
    wide, wide64 = dev(r.standard_normal((T, K + 11)), "bf16")
    w, w64 = dev(r.standard_normal((N, K)), "bf16")
    x64 = wide64[:, off:off + K]
    y = kda.linear(wide[:, off:off + K], w, out_dtype=torch.float32)
    no_error()
    check("y", y, x64 @ w64.T, product_tol(x64, w64.T, K, "bf16"))


@pytest.mark.parametrize("off,pad", [(0, 8), (8, 24), (1, 3), (3, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_column_blocks(off, pad, dtype):
    """Operands that are column blocks of wider arrays, aligned and not."""
    def view(t):
        wide = torch.full((t.shape[0], t.shape[1] + off + pad), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, off:off + t.shape[1]] = t
        return wide[:, off:off + t.shape[1]]
    linear_case(4, 70, 96, 56, dtype, act="gelu", bias=True, res=dtype, views=view)


def test_linear_in_place_residual_and_rows_behind():
    """y may be the residual itself, and rows and columns outside y keep their contents."""
    r = rng(5)
    x, x64 = dev(r.standard_normal((130, 64)), "bf16")
    w, w64 = dev(r.standard_normal((72, 64)), "bf16")
    buf = torch.full((140, 90), 7.0, device=DEV)
    res64 = r.standard_normal((130, 72))
    buf[:130, 8:80] = torch.from_numpy(res64).to(DEV)
    out = buf[:130, 8:80]
    kda.linear(x, w, residual=out, out=out, scale=0.25)
    no_error()
    ref = ol.linear(x64, w64, None, "none", res64.astype(np.float32).astype(np.float64), 0.25)[0]
    check("y", out, ref, product_tol(x64, w64.T, 64, "bf16") + 4 * U * np.abs(ref))
    b = buf.cpu()
    assert (b[130:] == 7).all() and (b[:, :8] == 7).all() and (b[:, 80:] == 7).all()


def test_linear_no_tokens():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones((40, 64), dtype=torch.bfloat16, device=DEV)
    y, z = kda.linear(x, w, save_pre_activation=True)
    dx, dw, db = kda.linear_bwd(x, w, y, need_bias=True)
    no_error()
    assert y.shape == z.shape == (0, 40) and dx.shape == (0, 64)
    assert not dw.any() and not db.any() and dw.shape == (40, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_wide_values(dtype):
    """Rows of very different sizes, and zero rows: errors stay relative to each sum's terms."""
    r = rng(6)
    T, K, N = 40, 160, 48
    x, x64 = dev(r.standard_normal((T, K)) * np.exp(r.uniform(-40, 40, (T, 1))), dtype)
    x[3] = 0
    x64[3] = 0
    w, w64 = dev(r.standard_normal((N, K)) * np.exp(r.uniform(-10, 10, (N, 1))), dtype)
    y = kda.linear(x, w, out_dtype=torch.float32)
    no_error()
    ref = x64 @ w64.T
    check("y", y, ref, product_tol(x64, w64.T, K, dtype))
    assert not y[3].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_infinite_token_stays_in_its_row(dtype):
    r = rng(7)
    x, _ = dev(r.standard_normal((150, 64)), dtype)
    w, _ = dev(r.standard_normal((64, 64)), dtype)
    clean = kda.linear(x, w)
    x[5, 9] = float("inf")
    x[77, 0] = float("nan")
    y = kda.linear(x, w)
    no_error()
    keep = [t for t in range(150) if t not in (5, 77)]
    assert torch.equal(y[keep], clean[keep])
    assert not torch.isfinite(y[5]).any() and torch.isnan(y[77]).all()


def test_linear_repeats_bit_for_bit():
    r = rng(8)
    x, _ = dev(r.standard_normal((900, 512)), "bf16")
    w, _ = dev(r.standard_normal((96, 512)), "bf16")
    dy, _ = dev(r.standard_normal((900, 96)), "bf16")
    first = (kda.linear(x, w),) + kda.linear_bwd(x, w, dy, need_bias=True)
    for _ in range(3):
        again = (kda.linear(x, w),) + kda.linear_bwd(x, w, dy, need_bias=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ----------------------------------------------------------------------------------- residual_norm

def residual_case(seed, T, N, dtype, h_dtype, *, res=True, post=False, gate=None, scale=1.0,
                  shift=0, weight=True, d_h=True, eps=1e-6):
    r = rng(seed, T, N)

    def arr(a, dt):
        t, v = dev(a, dt)
        if shift:                                      # not 16-byte aligned
            flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
            flat[shift:] = t.reshape(-1)
            t = flat[shift:].view(t.shape)
        return t, v
    x, x64 = arr(r.standard_normal((T, N)), dtype)
    rs, rs64 = arr(r.standard_normal((T, N)) * 2, h_dtype) if res else (None, None)
    w, w64 = arr(1 + 0.1 * r.standard_normal(N), "f32") if weight else (None, None)
    pw, pw64 = arr(1 + 0.1 * r.standard_normal(N), "f32") if post else (None, None)
    g, g64 = (None, None) if gate is None else arr(
        r.standard_normal(N if gate == "channel" else (T, N)), "f32" if gate == "channel" else dtype)
    y, h = kda.residual_norm(x, w, residual=rs, post_weight=pw, gate=g, scale=scale, eps=eps)
    no_error()
    y_ref, h_ref = ol.residual_norm(x64, w64, rs64, pw64, g64, scale, eps)
    terms = np.abs(h_ref - (rs64 if res else 0)) + (np.abs(rs64) if res else 0)
    check("h", h, h_ref, 64 * U * terms)
    if weight:
        check("y", y, y_ref, 128 * U * terms * ol.rms(h_ref, eps)[1] * np.abs(w64) + 64 * U * np.abs(y_ref))
    else:
        assert y is None

    hd = h_dtype if res else dtype
    dy, dy64 = arr(r.standard_normal((T, N)), dtype) if weight else (None, None)
    dh, dh64 = arr(r.standard_normal((T, N)), hd) if d_h else (None, None)
    h64 = host(h)
    dx, dres, dw, dpw, dg = kda.residual_norm_bwd(x, h, w, dy, dh, post_weight=pw, gate=g,
                                                  scale=scale, eps=eps)
    no_error()
    ref = ol.residual_norm_bwd(x64, h64, w64, dy64, dh64, pw64, g64, scale, eps)
    # absolute sums behind each gradient: r (|d| + |n| mean|d n|), plus d_h
    tot = np.abs(dh64) if d_h else np.zeros((T, N))
    if weight:
        n, rr = ol.rms(h64, eps)
        d = np.abs(dy64 * w64)
        tot = tot + rr * (d + np.abs(n) * np.mean(d * np.abs(n), -1, keepdims=True))
        check("d_weight", dw, ref[2], (T + 128) * U * np.abs(dy64 * n).sum(0))
    check("d_residual", dres, ref[1], 128 * U * tot)
    ag = 1 if g64 is None else np.abs(g64)
    u = np.abs(x64) if not post else np.abs(ol.rms(x64, eps)[0] * pw64)
    du = abs(scale) * tot * ag
    if gate == "token":
        check("d_gate", dg, ref[4], 256 * U * abs(scale) * tot * u)
    elif gate == "channel":
        check("d_gate", dg, ref[4].sum(0), (T + 256) * U * (abs(scale) * tot * u).sum(0))
    else:
        assert dg is None
    if post:
        n, rr = ol.rms(x64, eps)
        check("d_post_weight", dpw, ref[3], (T + 256) * U * (du * np.abs(n)).sum(0))
        d = du * np.abs(pw64)
        du = rr * (d + np.abs(n) * np.mean(d * np.abs(n), -1, keepdims=True))
    else:
        assert dpw is None
    check("dx", dx, ref[0], 512 * U * du)


@pytest.mark.parametrize("N", [1, 7, 8, 64, 100, 1000, 1024, 1032, 2048, 4095, 4096, 8192, 16383, 16384])
@pytest.mark.parametrize("T", [1, 5])
def test_residual_norm_widths(N, T):
    residual_case(1, T, N, "bf16", "bf16", post=True, gate="channel", scale=0.5)


@pytest.mark.parametrize("dtype,h_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("res", [False, True])
def test_residual_norm_forms(dtype, h_dtype, post, gate, res):
    residual_case(2, 37, 264, dtype, h_dtype, post=post, gate=gate, res=res, scale=0.7)


@pytest.mark.parametrize("weight,d_h", [(False, True), (True, False)])
def test_residual_norm_without_weight_or_stream_gradient(weight, d_h):
    residual_case(3, 20, 320, "bf16", "f32", post=True, gate="channel", weight=weight, d_h=d_h)


@pytest.mark.parametrize("N", [256, 129])
def test_residual_norm_unaligned(N):
    residual_case(4, 9, N, "bf16", "bf16", post=True, gate="token", shift=1)
    residual_case(4, 9, N, "f32", "f32", post=True, gate="token", shift=1)


@pytest.mark.parametrize("T,N", [(7500, 96), (2000, 2048), (1000, 4096), (470, 8200), (460, 16384)])
@pytest.mark.parametrize("dtype,h_dtype,post,gate", [
    ("bf16", "bf16", True, "token"), ("bf16", "f32", True, "channel"), ("f32", "f32", False, None),
    ("bf16", "bf16", False, "token")])
def test_residual_norm_many_rows(T, N, dtype, h_dtype, post, gate):
    """Enough rows that each CTA walks several of them through its ring."""
    residual_case(5, T, N, dtype, h_dtype, post=post, gate=gate, scale=0.5)


def test_residual_norm_zero_rows_and_no_tokens():
    x = torch.zeros((3, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    y, h = kda.residual_norm(x, w, residual=x)
    dx, dr, dw, _, _ = kda.residual_norm_bwd(x, h, w, torch.ones_like(x))
    e = torch.empty((0, 64), device=DEV)
    ye, he = kda.residual_norm(e, w, residual=e)
    g = torch.ones(64, device=DEV)
    out = kda.residual_norm_bwd(e, he, w, ye, post_weight=w, gate=g)
    no_error()
    assert not y.any() and not dw.any()
    assert torch.allclose(dr, torch.full_like(dr, 1e3)) and torch.equal(dx, dr)   # 1 / sqrt(eps)
    assert all(not t.any() for t in out[2:]) and out[0].shape == (0, 64)


def test_residual_norm_in_place_stream():
    r = rng(6)
    x, x64 = dev(r.standard_normal((40, 512)), "bf16")
    h, h64 = dev(r.standard_normal((40, 512)), "f32")
    w, w64 = dev(1 + 0.1 * r.standard_normal(512), "f32")
    y, h2 = kda.residual_norm(x, w, residual=h, h_out=h, scale=0.5)
    no_error()
    assert h2 is h
    y_ref, h_ref = ol.residual_norm(x64, w64, h64, None, None, 0.5)
    t = np.abs(h64) + np.abs(x64)
    check("h", h, h_ref, 64 * U * t)
    check("y", y, y_ref, 128 * U * t * ol.rms(h_ref, 1e-6)[1] * w64 + 64 * U * np.abs(y_ref))


def test_residual_norm_gate_column_block():
    r = rng(7)
    x, x64 = dev(r.standard_normal((33, 128)), "bf16")
    wide, wide64 = dev(r.standard_normal((33, 400)), "bf16")
    w, w64 = dev(1 + 0.1 * r.standard_normal(128), "f32")
    for off in (128, 131):
        y, h = kda.residual_norm(x, w, residual=x, gate=wide[:, off:off + 128])
        no_error()
        _, h_ref = ol.residual_norm(x64, w64, x64, None, wide64[:, off:off + 128])
        check("h", h, h_ref, 64 * U * (np.abs(x64) + np.abs(h_ref - x64)))


# -------------------------------------------------------------------------------------- gated_norm

def gated_case(seed, T, H, D, o_dtype, g_dtype, y_dtype, act, view=lambda t: t):
    r = rng(seed, T, H, D)
    o, o64 = dev(r.standard_normal((T, H, D)) * 0.2, o_dtype)
    g, g64 = dev(r.standard_normal((T, H, D)) * 2, g_dtype)
    w, w64 = dev(1 + 0.1 * r.standard_normal(D), "f32")
    dy, dy64 = dev(r.standard_normal((T, H, D)), y_dtype)
    g = view(g)
    y = kda.gated_norm(o, g, w, activation=act, out_dtype=DT[y_dtype])
    d_o, dg, dw = kda.gated_norm_bwd(o, g, w, dy, activation=act)
    no_error()
    n, rr = ol.rms(o64, 1e-6)
    a = np.abs(ol.act(act, g64))
    check("y", y, ol.gated_norm(o64, g64, w64, act), 96 * U * np.abs(n * w64) * np.maximum(a, np.abs(g64) if act == "silu" else a))
    ro, rg, rw = ol.gated_norm_bwd(o64, g64, w64, dy64, act)
    d = np.abs(dy64) * a
    dwn = d * np.abs(w64)
    check("d_o", d_o, ro, 256 * U * rr * (dwn + np.abs(n) * np.mean(dwn * np.abs(n), -1, keepdims=True)))
    slope = 1 + np.abs(g64) if act == "silu" else 1
    check("d_gate", dg, rg, 128 * U * np.abs(dy64 * n * w64) * slope)
    check("d_weight", dw, rw, (T * H + 256) * U * (d * np.abs(n)).reshape(-1, D).sum(0))


@pytest.mark.parametrize("D", [1, 8, 16, 37, 64, 100, 128, 136, 256, 257, 512, 1000, 1024])
@pytest.mark.parametrize("T,H", [(1, 1), (19, 3)])
def test_gated_norm_head_sizes(D, T, H):
    gated_case(1, T, H, D, "f32", "bf16", "bf16", "sigmoid")


@pytest.mark.parametrize("o", ["f32", "bf16"])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["sigmoid", "silu", "none"])
def test_gated_norm_types(o, g, y, act):
    gated_case(2, 33, 4, 128, o, g, y, act)


def test_gated_norm_many_rows():
    gated_case(3, 3000, 8, 16, "f32", "bf16", "bf16", "silu")


@pytest.mark.parametrize("off", [256, 3])
def test_gated_norm_packed_gate(off):
    def view(t):
        T, H, D = t.shape
        wide = torch.full((T, H * D + off + 5), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, off:off + H * D] = t.reshape(T, H * D)
        return wide[:, off:off + H * D].view(T, H, D)
    gated_case(4, 21, 2, 128, "f32", "bf16", "bf16", "silu", view)


def test_gated_norm_edges():
    """A zero row is zero; gates at the infinities; no tokens."""
    o = torch.ones((2, 1, 128), device=DEV)
    o[1] = 0
    g = torch.zeros((2, 1, 128), device=DEV)
    g[0, 0, 0], g[0, 0, 1] = float("inf"), float("-inf")
    w = torch.ones(128, device=DEV)
    y = kda.gated_norm(o, g, w)
    s = kda.gated_norm(o, g, w, activation="silu")
    d_o, dg, dw = kda.gated_norm_bwd(o, g, w, torch.ones_like(o))
    e = torch.empty((0, 2, 128), device=DEV)
    ye = kda.gated_norm(e, e, w)
    de = kda.gated_norm_bwd(e, e, w, ye)
    no_error()
    assert abs(y[0, 0, 0].item() - 1) < 1e-6 and y[0, 0, 1].item() == 0 and not y[1].any()
    assert s[0, 0, 0].item() == float("inf") and s[0, 0, 1].item() == 0
    assert torch.isfinite(d_o).all() and dg[0, 0, 0].item() == 0 and dg[0, 0, 1].item() == 0
    assert ye.shape == (0, 2, 128) and not de[2].any()


def test_norm_gradients_repeat_bit_for_bit():
    r = rng(8)
    x, _ = dev(r.standard_normal((700, 2048)), "bf16")
    w, _ = dev(r.standard_normal(2048), "f32")
    o = x.float().view(700, 16, 128)
    first = kda.residual_norm_bwd(x, x, w, x, x, post_weight=w, gate=w)
    fg = kda.gated_norm_bwd(o, o, w[:128].contiguous(), o)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in
                   zip(first, kda.residual_norm_bwd(x, x, w, x, x, post_weight=w, gate=w)))
        assert all(torch.equal(a, b) for a, b in zip(fg, kda.gated_norm_bwd(o, o, w[:128].contiguous(), o)))
