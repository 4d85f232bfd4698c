"""The key-value cache on the GPU where a caller's data are at the edge of what it may hold: tables whose pages
the references call free, entries and lengths that are out of range, values near
the end of fp32's range, pools of any order of their dimensions.

Tolerances as in `test_gpu_cache.py`: E for the scores, (n / 16 + 64) 2 U for sums, 2 (E + 2^-21) for weights.
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


def rng(*seed):
    return np.random.Generator(np.random.PCG64([*seed]))


def dev(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DT[dtype])
    return t.to(DEV), t.double().numpy()


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def host(t):
    return t.double().cpu().numpy()


def no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def error():
    torch.cuda.synchronize()
    return kda.get_device_error()


def close(name, got, ref, tol):
    """Element by element, beside half a step of the stored type."""
    g = host(got)
    half = torch.finfo(got.dtype).eps / 2
    lim = np.broadcast_to(tol, ref.shape)
    lim = lim + half * (np.abs(ref) + lim) + 1e-37
    assert np.array_equal(np.isfinite(g), np.isfinite(ref)), f"{name}: finite elsewhere"
    fine = np.isfinite(ref)
    assert np.array_equal(g[~fine], ref[~fine], equal_nan=True), name
    off = np.abs(g[fine] - ref[fine]) / lim[fine]
    assert np.all(off <= 1), f"{name}: off by {off.max()} of what it may be"


def reference(q64, k, v, W, out, D, **kw):
    """o, lse and their tolerances for one sequence."""
    ref, rl, mass, big, prod = oc.attention(q64, k, v, W, D ** -0.5, **kw)
    E = 2 * D * U * prod + 8 * U * (1 + big) + 2.0 ** -21
    sums = (len(k) / 16 + 64) * 2 * U
    tol = (2 * E + sums + (2.0 ** -16 if out == torch.bfloat16 else 0))[..., None] * mass
    seen = np.isfinite(rl)
    return ref, rl, tol, np.where(seen, E + sums + 4 * U * np.abs(np.where(seen, rl, 0)), 0)


# ------------------------------------------------------------------------------------------ tables

def refused(table, lens, refs, parent, new, P):
    got = kda.cache_update(ints(table), ints(lens), ints(refs), None if parent is None else ints(parent), ints(new), page_size=P)
    assert error() == _lib.KDA_DEVERR_PAGE
    assert torch.all(got.table == -1) and not got.lens.any() and not got.kept.any()
    assert torch.equal(got.refs, ints(refs)) and torch.all(got.src == -1) and torch.all(got.dst == -1)
    no_error()


@pytest.mark.parametrize("parent,new,free", [
    ([0, 0, 1], [7, 6, 6], 0),                 # a full page that both continuations of its row share
    ([0, 1, 1], [7, 6, 6], 2),
    ([0, 1, 1, 1], [8, 6, 6, 5], 2),
    ([0, 0, 0, 1], [8, 8, 3, 5], 1),           # full for two of them, not kept by the third
    ([0, 0, 1], [7, 6, 6], 1),                 # the page that they end inside
    ([0, 1], [8, 5], 3),                       # rows that only go on
    ([-1, 1, 1], [4, 5, 5], 0),                # a row that ends
])
def test_update_refuses_a_free_page_of_any_row(parent, new, free):
    refs = np.array([1, 1, 1, 1, 0, 0, 0, 0, 0, 0], np.int32)
    refs[free] = 0
    refused(np.array([[0, 1], [2, 3]], np.int32), [8, 5], refs, parent, new, 4)


def test_update_refuses_a_free_page_whose_changes_cancel():
    """One row that names it ends, another one forks."""
    refused(np.array([[0, 1], [0, 3]], np.int32), [8, 5], [0, 1, 1, 1, 0, 0, 0, 0], [-1, 1, 1], [0, 5, 5], 4)


@pytest.mark.parametrize("bad", [-2, -2 ** 31, 2, 2 ** 31 - 1])
@pytest.mark.parametrize("at", [0, 2])
def test_update_refuses_a_parent_out_of_range(bad, at):
    """-1 is the one that stands for nothing."""
    parent = [0, 1, -1]
    parent[at] = bad
    refused(np.array([[0, 1], [2, 3]], np.int32), [8, 5], [1, 1, 1, 1, 0, 0, 0, 0], parent, [8, 5, 3], 4)


@pytest.mark.parametrize("S", [4096, 4097, 6000])
@pytest.mark.parametrize("fork", [False, True])
@pytest.mark.parametrize("page", [0, 1])
def test_update_refuses_a_free_page_of_many_rows(S, fork, page):
    """One row of thousands names a free page; page 0 of it is full, page 1 the one that it ends inside."""
    table = np.arange(2 * S, dtype=np.int32).reshape(S, 2)
    refs = np.concatenate([np.ones(2 * S), np.zeros(50)]).astype(np.int32)
    parent = np.arange(S)
    if fork:
        parent[5] = 17
    new = np.full(S, 6)
    got, ref = kda.cache_update(ints(table), ints([5] * S), ints(refs), ints(parent), ints(new), page_size=4), \
        oc.update(table, [5] * S, refs, parent, new, 4)
    no_error()
    assert np.array_equal(got.table.cpu().numpy(), ref[0]) and np.array_equal(got.refs.cpu().numpy(), ref[2])
    refs[table[17, page]] = 0
    refused(table, [5] * S, refs, parent, new, 4)


@pytest.mark.parametrize("what", ["pages", "rows", "host"])
def test_pools_are_looked_at_before_anything_is_written(what):
    pool = {"pages": torch.zeros((7, 4), device=DEV), "rows": torch.zeros((8, 4), device=DEV)[:, ::2],
            "host": torch.zeros((8, 4))}[what]
    table, lens, refs = ints([[0, 1], [2, 3]]), ints([8, 5]), ints([1, 1, 1, 1, 0, 0, 0, 0])
    rows = kda.CacheRows(*(torch.full(s, 99, dtype=torch.int32, device=DEV) for s in ((2, 2), (2,), (8,), (2,), (2,), (2,))))
    with pytest.raises(ValueError):
        kda.cache_update(table, lens, refs, None, lens, page_size=4, pools=[pool], out=rows)
    moves = kda.CacheMoves(*(torch.full(s, 99, dtype=torch.int32, device=DEV) for s in ((2, 2), (8,), (8,), (4,), (4,))))
    with pytest.raises(ValueError):
        kda.cache_compact(table, lens, refs, page_size=4, pools=[pool], out=moves)
    torch.cuda.synchronize()
    assert all(torch.all(t == 99) for t in (*rows, *moves))
    no_error()


# --------------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("entry", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1, 9])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_attention_over_a_bad_page_reads_zeros(entry, at, dtype):
    r = rng(1)
    lens, P, D = [30, 41, 30], 16, 32
    table = np.array([[0, 1, -1], [2, 3, 4], [5, 6, -1]], np.int32)
    (kp, k64), (vp, v64) = (dev(r.standard_normal((9, P, 1, D)), dtype) for _ in range(2))
    q, q64 = dev(r.standard_normal((3, 2, D)), dtype)
    good, gl = kda.cache_attention(q, kp, vp, ints(table), ints(lens), return_lse=True)
    no_error()
    bad = table.copy()
    bad[1, at] = entry
    o, l = kda.cache_attention(q, kp, vp, ints(bad), ints(lens), return_lse=True)
    assert error() == _lib.KDA_DEVERR_PAGE
    k64, v64 = (x[[2, 3, 4]].copy() for x in (k64, v64))
    k64[at], v64[at] = 0, 0
    ref, rl, tol, ltol = reference(q64[1:2], k64.reshape(-1, 1, D)[:41], v64.reshape(-1, 1, D)[:41], 1, o.dtype, D)
    close("o", o[1:2], ref, tol)
    close("lse", l[1:2], rl, ltol)
    assert torch.equal(o[[0, 2]], good[[0, 2]]) and torch.equal(l[[0, 2]], gl[[0, 2]])
    no_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 4])
@pytest.mark.parametrize("length", [49, 1000, 2 ** 31 - 1, -1, -2 ** 31])
def test_a_length_out_of_range_is_an_empty_sequence(length, W, dtype):
    r = rng(2)
    lens, P, D = [30, 41, 30], 16, 32
    table = np.array([[0, 1, -1], [2, 3, 4], [5, 6, -1]], np.int32)
    kp, vp = (dev(r.standard_normal((9, P, 1, D)), dtype)[0] for _ in range(2))
    q, _ = dev(r.standard_normal((3 * W, 2, D)), dtype)
    good, gl = kda.cache_attention(q, kp, vp, ints(table), ints(lens), window=W, return_lse=True)
    no_error()
    o, l = kda.cache_attention(q, kp, vp, ints(table), ints([30, length, 30]), window=W, return_lse=True)
    assert error() == _lib.KDA_DEVERR_PAGE
    assert not o[W:2 * W].any() and torch.all(l[W:2 * W] == -float("inf"))
    keep = [i for i in range(3 * W) if i // W != 1]
    assert torch.equal(o[keep], good[keep]) and torch.equal(l[keep], gl[keep])
    no_error()


def test_attention_weights_of_later_keys_do_not_overflow():
    """A first block sets the running maximum, a key 9.9 powers of two above it follows: values of 1e36 stay finite."""
    D = 64
    for dtype in ("bf16", "f32"):
        k, v = np.zeros((200, 1, D)), np.full((200, 1, D), 1e36)
        k[150, 0, 0] = 9.9 * np.log(2) * D ** 0.5
        q = np.zeros((1, 2, D))
        q[..., 0] = 1
        compare(dtype, q, k, v, 1)


def compare(dtype, q, k, v, W, out=None, P=16, plant=None, **kw):
    """One sequence whose page table is in order, against fp64."""
    n, HK, D = k.shape
    pages = max(1, -(-n // P))
    room = [np.zeros((pages * P, HK, D)) for _ in range(2)]
    for x, y in zip(room, (k, v)):
        x[:n] = y
    (kp, k64), (vp, v64) = (dev(x.reshape(pages, P, HK, D), dtype) for x in room)
    k64, v64 = (x.reshape(-1, HK, D)[:n] for x in (k64, v64))
    if plant:
        plant(kp, vp)
    q, q64 = dev(q, dtype)
    o, l = kda.cache_attention(q, kp, vp, ints(np.arange(pages)[None]), ints([n]), window=W, out_dtype=DT[out or dtype],
                               return_lse=True, **kw)
    no_error()
    ref, rl, tol, ltol = reference(q64, k64, v64, W, o.dtype, D, **kw)
    # where weights are scaled by 2^-33, maxima are raised and log2 of the sums lowered by 33: both rounded to 2^-19
    close("o", o, ref, tol + 2.0 ** -19 * np.abs(v64).max())
    close("lse", l, rl, ltol + 2.0 ** -18)
    return o, l


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,H,HK,W,D", [(1, 1, 1, 1, 64), (40, 2, 1, 1, 64), (700, 2, 2, 1, 128), (6000, 4, 1, 1, 64),
                                        (900, 4, 2, 4, 128), (500, 12, 1, 1, 128), (500, 8, 1, 8, 64), (300, 4, 1, 2, 256),
                                        (300, 8, 1, 3, 256), (20000, 1, 1, 1, 32)])
@pytest.mark.parametrize("top", [1e35, 3e37, 2e38])
def test_attention_of_values_near_the_end_of_the_range(top, n, H, HK, W, D, dtype, out):
    """Sums of many such values pass the range, their weighted means do not: of one sign (the sums grow with every key)
    and of both, with a span, a cap and scores that rise."""
    r = rng(3, n, H, D)
    q, k = r.standard_normal((W, H, D)), r.standard_normal((n, HK, D))
    v = top * r.uniform(0.5, 1, (n, HK, D))
    compare(dtype, q, k, v, W, out)
    compare(dtype, q, k, v * r.choice([-1, 1], v.shape), W, out, span=max(1, n // 2), softcap=4.0)
    k += np.linspace(0, 3, n)[:, None, None] * q[:1, :1]
    compare(dtype, q, k, v, W, out)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_attention_of_large_values_beside_small_ones_and_hidden_infinities(dtype, out):
    """A few large values where most are small, in channels of their own, and infinite ones behind the end and in a
    draft's own row: the other channels and rows keep their accuracy."""
    r = rng(4)
    n, D, W = 3000, 64, 3
    q, k, v = r.standard_normal((W, 2, D)), r.standard_normal((n, 1, D)), r.standard_normal((n, 1, D))
    v[::7, 0, 5] = 1e38

    def behind(kp, vp):
        vp.view(-1, 1, D)[n:] = float("inf")
        kp.view(-1, 1, D)[n:] = float("nan")
    compare(dtype, q, k, v, W, out, plant=behind)
    o, l = compare(dtype, q, k, v, W, out)

    def last(kp, vp):
        vp.view(-1, 1, D)[n - 1] = float("inf")
    with pytest.raises(AssertionError, match="finite elsewhere"):
        compare(dtype, q, k, v, W, out, plant=last)
    pages = -(-n // 16)
    kp, vp = (torch.zeros((pages * 16, 1, D), dtype=DT[dtype], device=DEV) for _ in range(2))
    kp[:n], vp[:n] = dev(k, dtype)[0], dev(v, dtype)[0]
    vp[n - 1] = float("inf")
    a, b = kda.cache_attention(dev(q, dtype)[0], kp.view(pages, 16, 1, D), vp.view(pages, 16, 1, D), ints(np.arange(pages)[None]),
                               ints([n]), window=W, out_dtype=DT[out], return_lse=True)
    half = torch.finfo(a.dtype).eps / 2
    mean = np.abs(v).max(axis=(0, 1))          # the same products in another order, of weights that are scaled
    assert np.all(np.abs(host(a[:-1]) - host(o[:-1])) <= 2 * half * np.abs(host(o[:-1])) + 2.0 ** -14 * mean)
    assert torch.all(a[-1] == float("inf")) and torch.allclose(b, l, rtol=0, atol=2.0 ** -16)
    no_error()


# -------------------------------------------------------------------------------------------- pools

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["NPHD", "NHPD", "HNPD", "PNHD", "PHND", "HPND"])
def test_pools_of_any_order_of_their_dimensions(order, dtype):
    r = rng(5)
    size = dict(N=7, P=8, H=2, D=32)
    back = [order.index(c) for c in "NPHD"]
    pools = [torch.from_numpy(r.standard_normal([size[c] for c in order]).astype(np.float32)).to(DEV, DT[dtype]).permute(back)
             for _ in range(2)]
    dense = [p.contiguous() for p in pools]
    table, start = ints([[0, 3, 6], [5, 2, -1]]), ints([19, 8])
    k, v = (dev(r.standard_normal((5, 2, 32)), dtype)[0] for _ in range(2))
    q = dev(r.standard_normal((5, 4, 32)), dtype)[0]
    f, _ = kda.rotary_frequencies(32, device=DEV)
    out = []
    for kp, vp in (pools, dense):
        y = kda.cache_append(q, k, v, f, kp, vp, table, start, input_row_offsets=ints([0, 3, 5]))
        out.append([y, kda.cache_attention(y[[2, 4]], kp, vp, table, ints([22, 10]))])
    no_error()
    assert all(torch.equal(a, b) for a, b in zip(*out)) and all(torch.equal(a, b) for a, b in zip(pools, dense))
