"""The key-value cache (rotary, cache_append, cache_attention) on the GPU against the fp64 reference of
`oracle/cache.py`.

Tolerances, element by element, from the arithmetic (U = 2^-24, R(t) half a step of the stored type):

  rotary     the angle is off by 2^-33 turns and the frequency's own rounding in fp64 (|p| f 2^-52, below
             2^-24 for |p| < 2^24); sincospif is good to 2 ulp: c and s are off by at most 4 U; two
             products and a sum add 3 U: 8 U m (|a| + |b|)
  scores     D products, exact for bf16, with sums that tensor cores may cut off: 2 D U sum|q k| scale (fp32
             products: U each, inside it); scale, cap (tanhf 2 ulp of a value up to its cap), bias
             and the maximum's subtraction: 8 U (1 + largest |s|).  Together E
  weights    e^(s - m) by ex2.approx (2^-22): off by E + 2^-21 relative
  o          sums of n weighted values in blocks: (n / 16 + 64) 2 U; two bf16 parts of the weights for a bf16 o:
             2^-16.  The denominator carries the weights' error too: 2 (E + 2^-21) in all, times
             sum p |v| / sum p
  lse        E + 2^-21 + (n / 16 + 64) 2 U + 4 U |lse|
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def R(t):
    return torch.finfo(t).eps / 2


def rng(*seed):
    return np.random.Generator(np.random.PCG64([*seed]))


def dev(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype])
    return t.to(DEV), t.double().numpy()


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def host(t):
    return t.double().cpu().numpy()


def check(name, got, ref, tol):
    g = host(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if g.size == 0:
        return
    lim = np.broadcast_to(tol, ref.shape)
    lim = lim + R(got.dtype) * (np.abs(ref) + lim) + 1e-37
    fine = np.isfinite(ref)
    assert np.array_equal(np.isfinite(g), fine), f"{name}: finite elsewhere"
    assert np.array_equal(g[~fine], ref[~fine], equal_nan=True), name
    off = np.abs(g[fine] - ref[fine])
    assert np.all(off <= lim[fine]), f"{name}: off by {np.max(off / lim[fine])} of what it may be"


def no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def page_error():
    torch.cuda.synchronize()
    with pytest.raises(Exception):
        if kda.get_device_error() == _lib.KDA_DEVERR_PAGE:
            raise RuntimeError
    assert kda.get_device_error() == 0


# ------------------------------------------------------------------------------------------ rotary

def rotary_tol(x, R_, interleaved, m):
    a = np.abs(x[..., :R_])
    partner = a.reshape(*a.shape[:-1], -1, 2)[..., ::-1].reshape(a.shape) if interleaved else np.roll(a, R_ // 2, -1)
    return np.concatenate([8 * U * abs(m) * (a + partner), np.zeros_like(x[..., R_:])], -1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,HK,D,R_", [(1, 1, 1, 2, 2), (5, 3, 1, 128, 128), (37, 4, 2, 64, 32), (9, 2, 2, 100, 50),
                                         (19, 5, 3, 37, 36), (300, 8, 2, 128, 64), (3, 1, 1, 1024, 1024), (7, 2, 1, 24, 12),
                                         (2, 3, 0, 48, 10), (11, 1, 1, 1023, 1022)])
def test_rotary(T, H, HK, D, R_, dtype, interleaved):
    r = rng(T, H, D, R_)
    (q, q64), (k, k64) = (dev(r.standard_normal((T, h, D)), dtype) for h in (H, HK))
    pos = r.integers(-5, 100000, T)
    f, _ = oc.frequencies(R_)
    ft = torch.tensor(f, device=DEV)
    layout = "interleaved" if interleaved else "half"
    for transpose, call in ((False, kda.rotary), (True, kda.rotary_bwd)):
        yq, yk = call(q, k if HK else None, ints(pos), ft, layout=layout, magnitude=1.25)
        for y, x in ((yq, q64), (yk, k64)):
            if y is not None:
                check("rotary", y, oc.rotary(x, pos, f, interleaved, 1.25, transpose), rotary_tol(x, R_, interleaved, 1.25))
    assert (yk is None) == (HK == 0)
    no_error()


def test_rotary_packed_rows_far_positions_in_place():
    T, H, HK, D = 70, 4, 2, 64
    x, x64 = dev(rng(1).standard_normal((T, (H + 2 * HK) * D + 8)), "bf16")
    q, k = x[:, :H * D].unflatten(1, (H, D)), x[:, H * D:(H + HK) * D].unflatten(1, (HK, D))
    pos = rng(2).integers(0, 2 ** 23, T)
    f, m = kda.rotary_frequencies(32, scaling="by_parts", factor=8.0, trained_length=4096, device=DEV)
    f64 = f.cpu().numpy()
    wide = torch.tensor(pos, device=DEV)                     # int64
    yq, yk = kda.rotary(q, k, wide, f, magnitude=m)
    q64, k64 = x64[:, :H * D].reshape(T, H, D), x64[:, H * D:(H + HK) * D].reshape(T, HK, D)
    check("q", yq, oc.rotary(q64, pos, f64, False, m), rotary_tol(q64, 32, False, m))
    check("k", yk, oc.rotary(k64, pos, f64, False, m), rotary_tol(k64, 32, False, m))
    assert yq.is_contiguous()
    tail = x[:, (H + HK) * D:].clone()
    a, b = kda.rotary(q, k, ints(pos), f, magnitude=m, q_out=q, k_out=k)
    assert a.data_ptr() == q.data_ptr() and torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(x[:, (H + HK) * D:], tail)            # what lies between the rows
    no_error()


def test_rotary_unaligned_rows():
    x, x64 = dev(rng(3).standard_normal((20, 3 * 32 + 5)), "bf16")
    q = x[:, 5:].unflatten(1, (3, 32))
    pos = np.arange(20) * 77
    f, _ = oc.frequencies(32)
    for interleaved in (False, True):
        y, _ = kda.rotary(q, None, ints(pos), torch.tensor(f, device=DEV), layout="interleaved" if interleaved else "half")
        x3 = x64[:, 5:].reshape(20, 3, 32)
        check("q", y, oc.rotary(x3, pos, f, interleaved), rotary_tol(x3, 32, interleaved, 1.0))


def test_rotary_every_position_of_a_long_context_is_as_good():
    """The angle of position p and of p - 1 differ by f: no drift up to 2^31 (f a binary fraction, so that p f is
    exact in fp64)."""
    pos = np.array([0, 1, 2 ** 20 + 3, 2 ** 30 + 1, 2 ** 31 - 1])
    f = np.array([1.0, 2.0 ** -20])
    x, x64 = dev(np.ones((5, 1, 4)), "f32")
    y, _ = kda.rotary(x, None, ints(pos), torch.tensor(f, device=DEV))
    # 1 / 2 pi in fp64: the angle's share of p 2^-53 turns
    check("far", y, oc.rotary(x64, pos, f), 16 * U + (pos * 2.0 ** -52 * 2 * np.pi)[:, None, None])


def test_rotary_gradient_is_the_adjoint():
    T, H, D = 33, 2, 64
    (q, q64), (d, d64) = (dev(rng(4, i).standard_normal((T, H, D)), "f32") for i in range(2))
    f, m = kda.rotary_frequencies(48, device=DEV)
    pos = ints(rng(5).integers(0, 5000, T))
    y, g = kda.rotary(q, None, pos, f, layout="interleaved")[0], kda.rotary_bwd(d, None, pos, f, layout="interleaved")[0]
    a, b = (host(y) * d64).sum(), (q64 * host(g)).sum()
    assert abs(a - b) <= 8 * U * 4 * np.abs(q64).sum() * np.abs(d64).max()


def test_rotary_of_nothing():
    f = torch.ones(4, dtype=torch.float64, device=DEV)
    e = torch.empty((0, 2, 8), device=DEV)
    y, z = kda.rotary(e, e, ints(np.zeros(0)), f)
    assert y.shape == z.shape == (0, 2, 8)


# ------------------------------------------------------------------------------------------ append

def paged(r, lens, P, dtype, HK, D, spare=3, by_heads=False, first=None):
    """Pools with random contents and a table for `lens` tokens a row (entries before first[b] are -1)."""
    pages = [-(-n // P) for n in lens]
    first = first or [0] * len(lens)
    N = sum(pages) + spare
    order = list(r.permutation(N))
    table = np.full((len(lens), max(1, max(pages, default=1))), -1, np.int32)
    for b, n in enumerate(pages):
        for j in range(first[b], n):
            table[b, j] = order.pop()
    shape = (N, HK, P, D) if by_heads else (N, P, HK, D)
    pools = []
    for _ in range(2):
        t, v = dev(r.standard_normal(shape), dtype)
        pools.append((t.transpose(1, 2), v.swapaxes(1, 2)) if by_heads else (t, v))
    return table, pools


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,D,R_,by_heads,interleaved", [(1, 16, 16, False, False), (16, 128, 64, False, True),
                                                         (7, 40, 20, True, False), (64, 37, 36, False, True),
                                                         (24, 64, 0, True, False)])
def test_append(P, D, R_, by_heads, interleaved, dtype):
    r = rng(P, D, R_)
    H, HK = 4, 2
    new, start = [3, 0, 65, 1, 20], [0, 9, 5, 130, 31]
    table, ((kp, k64), (vp, v64)) = paged(r, [a + b for a, b in zip(new, start)], P, dtype, HK, D, by_heads=by_heads)
    T = sum(new) + 6                                         # six rows of padding behind the last sequence
    (q, q64), (k, kn), (v, vn) = (dev(r.standard_normal((T, h, D)), dtype) for h in (H, HK, HK))
    f, _ = oc.frequencies(R_) if R_ else (None, 1.0)
    offsets = np.concatenate([[0], np.cumsum(new)])
    out = torch.full_like(q, 7.0)
    got = kda.cache_append(q, k, v, None if f is None else torch.tensor(f, device=DEV), kp, vp, ints(table), ints(start),
                           input_row_offsets=ints(offsets), layout="interleaved" if interleaved else "half",
                           magnitude=1.5, q_out=out)
    assert got is out
    pos = np.concatenate([np.arange(n) + s for n, s in zip(new, start)])
    turn = (lambda x: oc.rotary(x, pos, f, interleaved, 1.5)) if R_ else (lambda x: x)
    n = sum(new)
    tol = (lambda x: rotary_tol(x, R_, interleaved, 1.5)) if R_ else (lambda x: 0 * x)
    check("q", out[:n], turn(q64[:n]), tol(q64[:n]))
    assert torch.all(out[n:] == 7.0)
    kk, ktol, row = turn(kn[:n]), np.zeros_like(k64), 0
    for b, m in enumerate(new):
        for i in range(m):
            p = start[b] + i
            k64[table[b, p // P], p % P] = kk[row]
            ktol[table[b, p // P], p % P] = tol(kn[:n])[row]
            v64[table[b, p // P], p % P] = vn[row]
            row += 1
    check("k pages", kp, k64, ktol)
    assert np.array_equal(host(vp), v64)                     # every other row as it was
    no_error()


def test_append_decode_form_without_queries():
    r = rng(9)
    start = [0, 15, 16, 40]
    table, ((kp, k64), (vp, v64)) = paged(r, [s + 1 for s in start], 16, "bf16", 2, 32)
    (k, kn), (v, vn) = (dev(r.standard_normal((4, 2, 32)), "bf16") for _ in range(2))
    assert kda.cache_append(None, k, v, None, kp, vp, ints(table), ints(start)) is None
    for b, s in enumerate(start):
        k64[table[b, s // 16], s % 16], v64[table[b, s // 16], s % 16] = kn[b], vn[b]
    assert np.array_equal(host(kp), k64) and np.array_equal(host(vp), v64)
    no_error()


@pytest.mark.parametrize("what", ["page", "negative", "behind", "start"])
def test_append_bad_pages(what):
    r = rng(10)
    start = [3, 3]
    table, ((kp, k64), (vp, v64)) = paged(r, [4, 4], 4, "bf16", 1, 16)
    kbad, sbad = table.copy(), list(start)
    if what == "page":
        kbad[0, 0] = kp.shape[0]
    elif what == "negative":
        kbad[0, 0] = -1
    elif what == "behind":
        sbad[0] = 4                                          # the row has one page
    else:
        sbad[0] = -1
    (k, kn), (v, vn) = (dev(r.standard_normal((2, 1, 16)), "bf16") for _ in range(2))
    kda.cache_append(None, k, v, None, kp, vp, ints(kbad), ints(sbad))
    page_error()
    k64[table[1, 0], 3], v64[table[1, 0], 3] = kn[1], vn[1]   # the other sequence is written
    assert np.array_equal(host(kp), k64) and np.array_equal(host(vp), v64)


def test_append_bad_offsets():
    r = rng(11)
    table, ((kp, k64), (vp, _)) = paged(r, [8, 8], 4, "bf16", 1, 16)
    (k, _), (v, _) = (dev(r.standard_normal((4, 1, 16)), "bf16") for _ in range(2))
    kda.cache_append(None, k, v, None, kp, vp, ints(table), ints([0, 0]), input_row_offsets=ints([0, 2, 9]))
    torch.cuda.synchronize()
    with pytest.raises(Exception):
        if kda.get_device_error() == _lib.KDA_DEVERR_OFFSETS:
            raise RuntimeError
    assert np.array_equal(host(kp), k64)


# --------------------------------------------------------------------------------------- attention

def attention_case(seed, lens, H, HK, D, P, dtype="bf16", W=1, out=None, softcap=0.0, span=0, slopes=False,
                   scale=0.0, by_heads=False, plant=None, lse=True, packed=False):
    r = rng(seed, D, P, H)
    first = [max(0, n - W - span + 1) // P if span else 0 for n in lens]
    table, ((kp, k64), (vp, v64)) = paged(r, lens, P, dtype, HK, D, by_heads=by_heads, first=first)
    B = len(lens)
    q, q64 = dev(r.standard_normal((B * W, (H + (1 if packed else 0)) * D)), dtype)
    q, q64 = q[:, :H * D].unflatten(1, (H, D)), q64[:, :H * D].reshape(B * W, H, D)
    sl = r.random(H).astype(np.float32) * 0.1 if slopes else None
    if plant:
        plant(table, kp, vp)
    got = kda.cache_attention(q, kp, vp, ints(table), ints(lens), window=W, scale=scale, softcap=softcap, span=span,
                              slopes=None if sl is None else torch.from_numpy(sl).to(DEV),
                              out_dtype=DT[out] if out else None, return_lse=lse)
    o, l = got if lse else (got, None)
    assert o.dtype == DT[out or dtype]
    for b, n in enumerate(lens):
        lo = first[b] * P
        k, v = (np.stack([p[table[b, j // P], j % P] if j >= lo else np.zeros((HK, D)) for j in range(n)])
                if n else np.zeros((0, HK, D)) for p in (k64, v64))
        ref, rl, mass, big, prod = oc.attention(q64[b * W:(b + 1) * W], k, v, W, scale or D ** -0.5, softcap, span, sl)
        E = (2 * D * U * prod + 8 * U * (1 + np.maximum(big, softcap)))
        E = E + 2.0 ** -21
        sums = (n / 16 + 64) * 2 * U
        rows = slice(b * W, (b + 1) * W)
        check("o", o[rows], ref, (2 * E + sums + (2.0 ** -16 if o.dtype == torch.bfloat16 else 0))[..., None] * mass)
        if lse:
            seen = np.isfinite(rl)
            check("lse", l[rows], rl, np.where(seen, E + sums + 4 * U * np.abs(np.where(seen, rl, 0)), 0))
    no_error()
    return o, l


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200, 333]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 16, 64, 72, 80, 128, 136, 256])
def test_attention_head_sizes(D, dtype):
    attention_case(1, LENS, 4, 2, D, 16, dtype)


def test_attention_head_size_of_one_piece_f32():
    attention_case(2, LENS, 2, 1, 4, 16, "f32")
    attention_case(2, LENS, 3, 1, 100, 16, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,HK,W", [(1, 1, 1), (6, 6, 1), (8, 1, 1), (7, 1, 1), (16, 2, 2), (9, 1, 1), (20, 2, 3), (33, 1, 1),
                                    (4, 4, 5), (4, 2, 17), (8, 1, 8), (2, 1, 64)])
def test_attention_groups_and_windows(H, HK, W, dtype):
    """Every number of rows of a key head: one tile and several, for each split of the warps."""
    attention_case(3, [0, 1, W - 1, W, W + 1, 40, 130, 300], H, HK, 64, 16, dtype, W=W)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,HK,W,D", [(4, 2, 4, 128), (12, 1, 1, 128), (5, 1, 5, 256), (32, 1, 1, 256), (3, 1, 1, 256)])
def test_attention_rows_of_wide_heads(H, HK, W, D, dtype):
    attention_case(4, [0, W, 77, 260], H, HK, D, 16, dtype, W=W, softcap=20.0)


@pytest.mark.parametrize("P", [1, 3, 8, 24, 64, 256])
@pytest.mark.parametrize("by_heads", [False, True])
def test_attention_page_sizes(P, by_heads):
    attention_case(5, LENS, 4, 2, 64, P, by_heads=by_heads)
    attention_case(6, LENS, 2, 2, 32, P, "f32", by_heads=by_heads, W=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(softcap=5.0), dict(slopes=True), dict(span=1), dict(span=7), dict(span=64), dict(span=100000),
                                dict(scale=0.7), dict(scale=-0.2), dict(softcap=30.0, slopes=True, span=50),
                                dict(span=2 ** 31 - 1), dict(packed=True)])
@pytest.mark.parametrize("W", [1, 3])
def test_attention_options(kw, W, dtype):
    attention_case(7, LENS, 4, 2, 64, 16, dtype, W=W, **kw)


@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_attention_output_types(dtype, out):
    attention_case(8, LENS, 4, 2, 128, 16, dtype, out=out)
    attention_case(8, LENS, 4, 2, 128, 16, dtype, out=out, lse=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H,HK,W", [([9001], 2, 1, 1), ([1, 6000, 3, 0, 2000], 4, 2, 1), ([2500, 2501], 4, 2, 6)])
def test_attention_split_over_the_length(lens, H, HK, W, dtype):
    attention_case(9, lens, H, HK, 64, 16, dtype, W=W, slopes=True)


def test_attention_many_sequences():
    attention_case(10, [int(n) for n in rng(10).integers(0, 40, 700)], 2, 1, 16, 16)


def test_attention_large_scores_do_not_overflow():
    """Running maxima that jump up and down by hundreds."""
    r = rng(12)
    n, D = 600, 64
    table, ((kp, k64), (vp, v64)) = paged(r, [n], 16, "f32", 1, D)
    q, q64 = dev(r.standard_normal((1, 2, D)) * 40, "f32")
    o, l = kda.cache_attention(q, kp, vp, ints(table), ints([n]), return_lse=True)
    k, v = (np.stack([p[table[0, j // 16], j % 16] for j in range(n)]) for p in (k64, v64))
    ref, rl, mass, big, prod = oc.attention(q64, k, v, 1, D ** -0.5)
    E = 2 * D * U * prod + 8 * U * (1 + big) + 2.0 ** -21
    assert big.max() > 100
    check("o", o, ref, (2 * E + 200 * U)[..., None] * mass)
    check("lse", l, rl, E + 200 * U + 4 * U * np.abs(rl))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,H,W", [(64, 2, 1), (64, 4, 3), (128, 8, 3), (256, 4, 2)])
def test_attention_what_is_not_seen_does_not_reach(D, H, W, dtype, bad):
    """Planted behind a sequence's end in its own last page, in free pages, before the span, and in a draft's own keys
    and values for the queries before it."""
    lens, P = [5, 37, 130], 16

    def plant(table, kp, vp):
        for pool in (kp, vp):
            for b, n in enumerate(lens):
                if n % P:
                    pool[int(table[b, n // P]), n % P:] = bad
            pool[sorted(set(range(pool.shape[0])) - set(table[table >= 0].tolist()))] = bad
    attention_case(13, lens, H, 2, D, P, dtype, W=W, plant=plant)
    r = rng(14)
    span = 20
    table, ((kp, k64), (vp, v64)) = paged(r, lens, P, dtype, 2, D)
    q, q64 = dev(r.standard_normal((3 * W, H, D)), dtype)
    k0, v0 = kp.clone(), vp.clone()
    for b, n in enumerate(lens):
        for j in list(range(0, max(0, n - W - span + 1))) + ([n - 1] if W > 1 else []):
            kp[int(table[b, j // P]), j % P] = bad
            vp[int(table[b, j // P]), j % P] = bad
    a = kda.cache_attention(q, k0, v0, ints(table), ints(lens), window=W, span=span)
    c = kda.cache_attention(q, kp, vp, ints(table), ints(lens), window=W, span=span)
    keep = [b * W + w for b in range(3) for w in range(W - 1 if W > 1 else 1)]
    x, y = host(a)[keep], host(c)[keep]
    assert np.all(np.isfinite(y))
    # the same products, in another order where the values were added one by one
    assert np.all(np.abs(x - y) <= 2 * R(a.dtype) * np.abs(x) + 2.0 ** (-15 if dtype == "bf16" else -18) * np.abs(host(v0)).max())
    no_error()


def test_attention_a_draft_that_is_not_finite_spoils_its_own_row():
    r = rng(15)
    table, ((kp, _), (vp, _)) = paged(r, [40], 16, "bf16", 1, 64)
    q, _ = dev(r.standard_normal((2, 2, 64)), "bf16")
    vp[int(table[0, 2]), 7] = float("inf")
    o = kda.cache_attention(q, kp, vp, ints(table), ints([40]), window=2)
    assert torch.isfinite(o[0]).all() and not torch.isfinite(o[1]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_infinite_values_and_keys_that_are_seen(dtype):
    """An infinite value makes its channel infinite, of either sign; a key with infinite scores of the lower sign has
    no weight, of the higher one makes a NaN of the row."""
    r = rng(20)
    table, ((kp, k64), (vp, _)) = paged(r, [40], 16, dtype, 1, 64)
    q = torch.ones((1, 2, 64), dtype=DT[dtype], device=DEV)
    at = (int(table[0, 1]), 3)
    good = kda.cache_attention(q, kp, vp, ints(table), ints([40]))
    v = vp.clone()
    v[at][0, 5], v[at][0, 6] = float("inf"), float("-inf")
    o = kda.cache_attention(q, kp, v, ints(table), ints([40]))
    assert torch.all(o[..., 5] == float("inf")) and torch.all(o[..., 6] == -float("inf"))
    rest = [c for c in range(64) if c not in (5, 6)]
    # another order of the sums
    assert torch.allclose(o[..., rest].float(), good[..., rest].float(), rtol=2 * R(o.dtype), atol=2.0 ** -14)
    k = kp.clone()
    k[at][0, 9] = float("-inf")
    o, l = kda.cache_attention(q, k, vp, ints(table), ints([40]), return_lse=True)
    keep = [j for j in range(40) if j != 19]
    kk = np.stack([k64[table[0, j // 16], j % 16] for j in keep])
    vv = np.stack([host(vp)[table[0, j // 16], j % 16] for j in keep])
    ref, rl, mass, big, prod = oc.attention(host(q), kk, vv, 1, 0.125)
    E = 2 * 64 * U * prod + 8 * U * (1 + big) + 2.0 ** -21
    check("o", o, ref, (2 * E + 140 * U + 2.0 ** -16)[..., None] * mass)
    check("lse", l, rl, E + 140 * U + 4 * U * np.abs(rl))
    k[at][0, 9] = float("inf")
    assert torch.isnan(kda.cache_attention(q, k, vp, ints(table), ints([40]))).all()
    no_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_bad_pages_and_lengths(dtype):
    r = rng(16)
    lens, P = [30, 30, 30], 16
    table, ((kp, _), (vp, _)) = paged(r, lens, P, dtype, 1, 32)
    q, _ = dev(r.standard_normal((3, 2, 32)), dtype)
    good = kda.cache_attention(q, kp, vp, ints(table), ints(lens))
    for change in ("page", "negative", "long", "below"):
        t, n = table.copy(), list(lens)
        if change == "page":
            t[1, 1] = kp.shape[0]
        elif change == "negative":
            t[1, 0] = -1
        else:
            n[1] = 33 if change == "long" else -4            # a row has two pages
        o = kda.cache_attention(q, kp, vp, ints(t), ints(n))
        page_error()
        assert torch.equal(o[[0, 2]], good[[0, 2]]) and torch.isfinite(o).all()


def test_attention_repeats_bit_for_bit_and_lengths_may_be_uint32():
    r = rng(17)
    lens = [5000, 0, 77]
    table, ((kp, _), (vp, _)) = paged(r, lens, 16, "bf16", 2, 128)
    q, _ = dev(r.standard_normal((3, 4, 128)), "bf16")
    a = [kda.cache_attention(q, kp, vp, ints(table), ints(lens)) for _ in range(5)]
    n = ints(lens).view(torch.uint32) if hasattr(torch, "uint32") else ints(lens)
    a.append(kda.cache_attention(q, kp, vp, ints(table), n))
    assert all(torch.equal(a[0], x) for x in a[1:])


def test_attention_of_nothing():
    e = torch.empty((0, 2, 16), dtype=torch.bfloat16, device=DEV)
    pages = torch.zeros((1, 4, 1, 16), dtype=torch.bfloat16, device=DEV)
    o = kda.cache_attention(e, pages, pages, torch.empty((0, 1), dtype=torch.int32, device=DEV), ints(np.zeros(0)))
    assert o.shape == e.shape
    # a table without columns: every sequence is empty
    q = torch.ones((2, 2, 16), dtype=torch.bfloat16, device=DEV)
    o, l = kda.cache_attention(q, pages, pages, torch.empty((2, 0), dtype=torch.int32, device=DEV), ints([0, 0]), return_lse=True)
    assert not o.any() and torch.all(l == -float("inf"))
    no_error()


def test_attention_offsets_past_two_to_the_31():
    """Pages that lie more than 2^31 elements behind the pool's start."""
    N, P, HK, D = 2 ** 17 + 3, 16, 8, 128                    # 2^31 elements and a little, 4.3 GB
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    kp = torch.zeros((N, P, HK, D), dtype=torch.bfloat16, device=DEV)
    r = rng(18)
    k, k64 = dev(r.standard_normal((2, P, HK, D)), "bf16")
    kp[N - 2:] = k
    q, q64 = dev(r.standard_normal((1, HK, D)), "bf16")
    o = kda.cache_attention(q, kp, kp, ints([[N - 2, N - 1]]), ints([30]))
    flat = k64.reshape(2 * P, HK, D)[:30]
    ref, _, mass, big, prod = oc.attention(q64, flat, flat, 1, D ** -0.5)
    E = 2 * D * U * prod + 8 * U * (1 + big) + 2.0 ** -21
    check("o", o, ref, (2 * E + 130 * U + 2.0 ** -16)[..., None] * mass)
    v, vn = dev(r.standard_normal((1, HK, D)), "bf16")
    kda.cache_append(None, v, v, None, kp, kp.clone(), ints([[N - 2, N - 1]]), ints([30]))
    assert np.array_equal(host(kp[N - 1, 14]), vn[0])
    no_error()
