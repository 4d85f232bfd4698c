"""The key-value cache's entry points without a GPU: every refusal comes back before anything touches
CUDA."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib, build as kbuild, cache
from oracle import cache as oc

A = 1 << 20                       # an aligned address that is never read: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _lib.load()


def rotary_params(**kw):
    base = dict(tokens=10, num_q_heads=4, num_k_heads=2, head_dim=16, rot_dim=8, dtype=1, magnitude=1.0)
    base.update(kw)
    return _lib.KdaRotaryParams(**base)


def cache_params(**kw):
    base = dict(tokens=3, num_seqs=3, num_q_heads=4, num_kv_heads=2, head_dim=16, rot_dim=0, dtype=1,
                o_dtype=1, page_size=8, max_pages=5, num_pages=20, window=1, magnitude=1.0,
                page_stride=8 * 2 * 16, page_row_stride=2 * 16, page_head_stride=16)
    base.update(kw)
    return _lib.KdaCacheParams(**base)


def rows_params(**kw):
    base = dict(rows=3, rows_out=4, max_pages=5, page_size=8, num_pages=20)
    base.update(kw)
    return _lib.KdaCacheRowsParams(**base)


def test_struct_layouts():
    assert ctypes.sizeof(_lib.KdaRotaryParams) == 72
    assert _lib.KdaRotaryParams.magnitude.offset == 36 and _lib.KdaRotaryParams.q_row_stride.offset == 40
    assert ctypes.sizeof(_lib.KdaCacheParams) == 128
    assert _lib.KdaCacheParams.magnitude.offset == 60 and _lib.KdaCacheParams.page_stride.offset == 104
    assert ctypes.sizeof(_lib.KdaCacheRowsParams) == 20


@pytest.mark.parametrize("name", ["kda_rotary_fwd", "kda_rotary_bwd"])
def test_rotary_refusals(lib, name):
    def call(p=None, q=A, k=A, pos=A, f=A, qo=A, ko=A):
        return getattr(lib, name)(ctypes.byref(p or rotary_params()), q, k, pos, f, qo, ko, None)
    assert getattr(lib, name)(None, A, A, A, A, A, A, None) == INVALID
    assert call(p=rotary_params(tokens=0), q=None, k=None, pos=None, f=None, qo=None, ko=None) == OK
    assert call(p=rotary_params(num_q_heads=0, num_k_heads=0)) == OK
    for kw in (dict(tokens=-1), dict(num_q_heads=-1), dict(head_dim=0), dict(dtype=2), dict(rot_dim=0),
               dict(rot_dim=7), dict(rot_dim=18), dict(magnitude=float("nan")), dict(q_row_stride=63),
               dict(k_out_row_stride=-32)):
        assert call(p=rotary_params(**kw)) == INVALID, kw
    for kw in (dict(head_dim=1026), dict(num_q_heads=1 << 22), dict(tokens=1 << 31)):
        assert call(p=rotary_params(**kw)) == UNSUPPORTED, kw
    assert call(q=None) == INVALID and call(k=None) == INVALID and call(pos=None) == INVALID
    assert call(f=None) == INVALID and call(qo=None) == INVALID and call(ko=None) == INVALID
    assert call(q=A + 1) == INVALID and call(pos=A + 2) == INVALID and call(f=A + 4) == INVALID
    assert call(p=rotary_params(wide_positions=1), pos=A + 4) == INVALID


def test_append_refusals(lib):
    def call(p=None, q=A, k=A, v=A, f=None, kp=A, vp=A, table=A, start=A, off=None, qo=A):
        return lib.kda_cache_append(ctypes.byref(p or cache_params()), q, k, v, f, kp, vp, table, start, off, qo, None)
    assert call(p=cache_params(tokens=0, num_seqs=0), q=None, k=None, v=None) == OK
    for kw in (dict(num_seqs=-1), dict(num_kv_heads=0), dict(dtype=3), dict(page_size=0), dict(max_pages=-1),
               dict(rot_dim=3), dict(rot_dim=18), dict(magnitude=float("inf")), dict(page_head_stride=15),
               dict(page_row_stride=31), dict(page_stride=255), dict(page_stride=0), dict(v_row_stride=31),
               dict(tokens=4)):                                  # without offsets one token a sequence
        assert call(p=cache_params(**kw)) == INVALID, kw
    assert call(p=cache_params(head_dim=1026, page_head_stride=1026, page_row_stride=2052, page_stride=1 << 20)) == UNSUPPORTED
    assert call(p=cache_params(rot_dim=8)) == INVALID            # turned channels without frequencies
    assert call(f=A) == INVALID                                  # and the other way round
    for kw in (dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(table=None), dict(start=None),
               dict(q=None), dict(qo=None), dict(k=A + 1), dict(kp=A + 1), dict(table=A + 2), dict(off=A + 2)):
        assert call(**kw) == INVALID, kw


def test_attention_refusals(lib):
    n = ctypes.c_size_t(0)

    def size(**kw):
        return lib.kda_cache_attention_workspace_size(ctypes.byref(cache_params(**kw)), ctypes.byref(n))
    assert size() == OK and n.value > 0
    # pages by heads: [num_pages, HK, page_size, d]
    assert size(page_row_stride=16, page_head_stride=128) == OK
    for kw in (dict(num_q_heads=0), dict(num_q_heads=3), dict(o_dtype=2), dict(window=0), dict(span=-1),
               dict(scale=float("nan")), dict(softcap=-1.0), dict(softcap=float("inf")), dict(q_row_stride=60),
               dict(page_row_stride=36), dict(page_stride=260), dict(page_row_stride=16, page_head_stride=120)):
        assert size(**kw) == INVALID, kw
    for kw in (dict(window=65), dict(head_dim=264, page_head_stride=264, page_row_stride=528, page_stride=8 * 528),
               dict(head_dim=12), dict(max_pages=1 << 30, num_seqs=1 << 12)):
        assert size(**kw) == UNSUPPORTED, kw
    assert lib.kda_cache_attention_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.kda_cache_attention_workspace_size(ctypes.byref(cache_params()), None) == INVALID
    size()
    need = n.value

    def call(p=None, q=A, k=A, v=A, t=A, lens=A, sl=None, o=A, lse=None, ws=A, nb=need):
        return lib.kda_cache_attention(ctypes.byref(p or cache_params()), q, k, v, t, lens, sl, o, lse, ws, nb, None)
    assert call(p=cache_params(num_seqs=0), q=None, k=None) == OK
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(t=None), dict(lens=None), dict(o=None), dict(q=A + 8),
               dict(k=A + 4), dict(v=A + 2), dict(t=A + 2), dict(lens=A + 1), dict(sl=A + 2), dict(o=A + 1), dict(lse=A + 2)):
        assert call(**kw) == INVALID, kw
    assert call(ws=None) == WORKSPACE and call(nb=need - 1) == WORKSPACE and call(ws=A + 128) == WORKSPACE


def test_tables_refusals(lib):
    n = ctypes.c_size_t(0)

    def size(**kw):
        return lib.kda_cache_rows_workspace_size(ctypes.byref(rows_params(**kw)), ctypes.byref(n))
    assert size() == OK
    for kw in (dict(rows=-1), dict(rows_out=-1), dict(max_pages=-1), dict(page_size=0), dict(num_pages=-1)):
        assert size(**kw) == INVALID, kw
    assert size(num_pages=(1 << 28) + 1) == UNSUPPORTED and size(rows=(1 << 24) + 1) == UNSUPPORTED
    size()
    need = n.value

    def update(p=None, ws=A, nb=need, **kw):
        a = dict(table=A, lens=A, refs=A, parent=A, new=A, ot=A, ol=A, orf=A, kept=A, src=A, dst=A)
        a.update(kw)
        return lib.kda_cache_update(ctypes.byref(p or rows_params()), *a.values(), ws, nb, None)
    for name in ("table", "lens", "refs", "new", "ot", "ol", "orf", "kept", "src", "dst", "parent"):
        assert update(**{name: None}) == INVALID, name           # no parent: rows_out has to be rows
        assert update(**{name: A + 2}) == INVALID, name
    assert update(ws=None) == WORKSPACE and update(nb=need - 4) == WORKSPACE and update(ws=A + 4) == WORKSPACE

    def compact(ws=A, nb=need, **kw):
        a = dict(table=A, lens=A, refs=A, ot=A, orf=A, pm=A, src=A, dst=A)
        a.update(kw)
        return lib.kda_cache_compact(ctypes.byref(rows_params()), *a.values(), ws, nb, None)
    for name in ("table", "lens", "refs", "ot", "orf", "pm", "src", "dst"):
        assert compact(**{name: None}) == INVALID and compact(**{name: A + 1}) == INVALID, name
    assert compact(ws=None) == WORKSPACE and compact(nb=0) == WORKSPACE


def test_copy_refusals(lib):
    def call(pools=(A, A), size=(64, 64), stride=(64, 64), src=A, dst=A, n=4, pages=10, count=2):
        P, I = ctypes.c_void_p, ctypes.c_int64
        return lib.kda_cache_copy((P * 2)(*pools), (I * 2)(*size), (I * 2)(*stride), count, src, dst, n, pages, None)
    assert call(count=0) == OK and call(n=0) == OK and call(pages=0) == OK
    for kw in (dict(count=-1), dict(n=-1), dict(pages=-1), dict(src=None), dict(dst=None), dict(src=A + 1),
               dict(pools=(A, None)), dict(size=(64, -1)), dict(stride=(64, 63))):
        assert call(**kw) == INVALID, kw
    assert call(n=1 << 31) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x, f = torch.zeros(3, 2, 8), torch.zeros(4, dtype=torch.float64)
    pages, i = torch.zeros(5, 4, 2, 8), torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: kda.rotary(x, x, i, f), lambda: kda.rotary_bwd(x, None, i, f),
                 lambda: kda.cache_append(x, x, x, f, pages, pages, table, i),
                 lambda: kda.cache_attention(x, pages, pages, table, i),
                 lambda: kda.cache_update(table, i, i, None, i, page_size=4),
                 lambda: kda.cache_compact(table, i, i, page_size=4), lambda: kda.cache_copy([pages], i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    kda.cache_copy([], i, i)                                     # nothing to copy


@pytest.mark.parametrize("call", [
    lambda x, t: cache._heads(x[0], "x"),                                  # not [T, H, d]
    lambda x, t: cache._heads(x.half(), "x"),
    lambda x, t: cache._heads(x[:, :, ::2], "x"),
    lambda x, t: cache._heads(x.transpose(0, 1), "x"),
    lambda x, t: cache._heads(x[:1].expand(6, 4, 8), "x"),                 # rows over one another
    lambda x, t: cache._heads(x, "x", x[:3]),
    lambda x, t: cache._heads(x, "x", x.bfloat16()),
    lambda x, t: cache._layout("pairs"),
    lambda x, t: cache._frequencies(torch.zeros(4), 8),                    # not fp64
    lambda x, t: cache._frequencies(torch.zeros(5, dtype=torch.float64), 8),
    lambda x, t: cache._frequencies(torch.zeros(0, dtype=torch.float64), 8),
    lambda x, t: cache._place(x.transpose(0, 1), x, "out"),
    lambda x, t: cache._place(x.bfloat16(), x, "out"),
    lambda x, t: cache._pages(_lib.KdaCacheParams(), x[None], x[None].bfloat16(), t, 3),
    lambda x, t: cache._pages(_lib.KdaCacheParams(), x, x, t, 3),
    lambda x, t: cache._pages(_lib.KdaCacheParams(), x[None].expand(4, 6, 4, 8), x[None].expand(4, 6, 4, 8), t, 3),
    lambda x, t: cache._pages(_lib.KdaCacheParams(), x[None], x[None], t.long(), 3),
    lambda x, t: cache._pages(_lib.KdaCacheParams(), x[None], x[None], t, 4),
    lambda x, t: cache._pages(_lib.KdaCacheParams(), x[None], x[None], t[:, ::2], 3),
    lambda x, t: cache._index(t[0].long(), 2, "lens"),
    lambda x, t: cache._index(t[:, 0], 3, "lens"),
    lambda x, t: kda.rotary_frequencies(7, device="cpu"),
    lambda x, t: kda.rotary_frequencies(8, scaling="cubic", device="cpu"),
    lambda x, t: kda.rotary_frequencies(8, scaling="by_parts", factor=2.0, device="cpu"),
    lambda x, t: kda.rotary_frequencies(8, base=0.0, device="cpu"),
    lambda x, t: kda.rotary(x, x, t[:, 0], None),
])
def test_binding_checks(call):
    with pytest.raises(ValueError):
        call(torch.zeros(6, 4, 8), torch.zeros(3, 2, dtype=torch.int32))


def test_outputs_have_memory_of_their_own():
    x, f = torch.zeros(3, 2, 8), torch.zeros(4, dtype=torch.float64)
    pages, i = torch.zeros(5, 4, 2, 8), torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: kda.rotary(x, x.clone(), i, f, q_out=pages[0, :3], k_out=pages[0, :3]),
                 lambda: kda.cache_append(x, x.clone(), x.clone(), f, pages, pages, table, i, q_out=pages[0, :3]),
                 lambda: kda.cache_attention(x, pages, pages, table, i, out=x)):
        with pytest.raises(ValueError, match="memory of its own"):
            call()
    row = kda.CacheRows(table, i, i, i, i, i)
    with pytest.raises(ValueError, match="memory of its own"):
        cache._out(row, [(n, t.shape) for n, t in zip(row._fields, row)], (table,))


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="by_parts", factor=8.0, trained_length=4096),
                                dict(base=500000.0, scaling="by_parts", factor=16.0, trained_length=8192, slow=2.0, fast=20.0)])
@pytest.mark.parametrize("R", [2, 50, 128])
def test_frequencies(kw, R):
    f, m = kda.rotary_frequencies(R, device="cpu", **kw)
    ref, mr = oc.frequencies(R, **kw)
    assert f.dtype == torch.float64
    # a power and a few products in fp64
    assert np.allclose(f.numpy(), ref, rtol=1e-14, atol=0) and abs(m - mr) < 1e-15


@pytest.mark.parametrize("a,b", [("lens", "kept"), ("src", "dst"), ("kept", "dst")])
def test_one_tensor_for_two_outputs_is_refused(a, b):
    row = kda.CacheRows(*(torch.zeros(s, dtype=torch.int32) for s in ((3, 2), 3, 5, 3, 3, 3)))
    like = [(n, t.shape) for n, t in zip(row._fields, row)]
    inputs = (torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32), None)
    assert cache._out(row, like, inputs) is row
    with pytest.raises(ValueError, match="memory of its own"):
        cache._out(row._replace(**{a: getattr(row, b)}), like, inputs)


def test_outputs_that_overlap_by_a_shift_are_refused():
    """Blocks would write rows that others have not read yet; columns of one packed array that only alternate are apart."""
    f, i, table = torch.zeros(4, dtype=torch.float64), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    big, pages = torch.zeros(8, 2, 8), torch.zeros(5, 4, 2, 8)
    q, k, packed = big[:3], torch.zeros(3, 2, 8), torch.zeros(3, 9, 8)
    a, b, c = packed[:, :2], packed[:, 2:4], packed[:, 1:3]
    for call in (lambda: kda.rotary(q, None, i, f, q_out=big[1:4]), lambda: kda.rotary(k, q, i, f, k_out=big[2:5]),
                 lambda: kda.rotary_bwd(q, None, i, f, dq_out=big[1:4]), lambda: kda.rotary(a, b, i, f, q_out=c),
                 lambda: kda.rotary(a, b, i, f, q_out=b), lambda: kda.rotary(a, b, i, f, k_out=c),
                 lambda: kda.rotary(a, None, i, f, q_out=packed.view(-1)[:48].view(3, 2, 8)),
                 lambda: kda.rotary(k, k.clone(), i, f, q_out=q, k_out=big[1:4]),
                 lambda: kda.cache_append(q, k, k.clone(), f, pages, pages.clone(), table, i, q_out=big[1:4]),
                 lambda: kda.cache_append(k, k.clone(), k.clone(), f, pages, pages.clone(), table, i, q_out=pages[1, 1:]),
                 lambda: kda.cache_attention(q, pages, pages, table, i, out=big[1:4]),
                 lambda: kda.cache_attention(q, pages, pages, table, i, out=pages[4, 1:])):
        with pytest.raises(ValueError, match="memory of its own"):
            call()
    for call in (lambda: kda.rotary(q, k, i, f, q_out=q, k_out=big[3:6]), lambda: kda.rotary(a, b, i, f, q_out=a, k_out=b),
                 lambda: kda.rotary(a, b, i, f, q_out=packed[:, 4:6], k_out=packed[:, 7:9]),
                 lambda: kda.cache_attention(q, pages, pages, table, i, out=big[3:6])):
        with pytest.raises(ValueError, match="CUDA"):            # what comes next on the host
            call()
    room = torch.zeros(64, dtype=torch.int32)
    row = kda.CacheRows(room[:6].view(3, 2), room[6:9], room[9:14], room[14:17], room[17:20], room[20:23])
    like = [(n, t.shape) for n, t in zip(row._fields, row)]
    cache._out(row, like, (room[23:29], room[29:32], None, room[23:27]))
    for bad, inputs in ((row._replace(kept=room[8:11]), ()), (row, (room[22:25],)), (row, (room[13:14],)),
                        (row._replace(dst=room[19:22]), ()), (row, (room[0:64],))):
        with pytest.raises(ValueError, match="memory of its own"):
            cache._out(bad, like, inputs)


def test_one_pool_for_keys_and_values_is_refused(monkeypatch):
    """Two blocks would write one row.  The check of an append's pools comes behind those of its plan, made up here."""
    class Called(Exception):
        pass

    def called(*a):
        raise Called
    monkeypatch.setattr(cache, "_plan_append", lambda *a: cache._Plan("kda_cache_append", cache_params(), torch.device("cuda:0")))
    monkeypatch.setattr(cache, "_call", called)
    x, i, table = torch.zeros(3, 2, 8), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    both, by_row = torch.zeros(6, 4, 2, 8), torch.zeros(5, 4, 2, 2, 8)

    def append(kp, vp):
        kda.cache_append(None, x, x, None, kp, vp, table, i)
    for kp, vp in ((both, both), (both[1:], both[:-1]), (both[:, 1:], both[:, :-1]), (by_row[:, :, 0], by_row[:, :, 0])):
        with pytest.raises(ValueError, match="memory of its own"):
            append(kp, vp)
    for kp, vp in ((both, both.clone()), (by_row[:, :, 0], by_row[:, :, 1]), (by_row[:, :, :, 0], by_row[:, :, :, 1]),
                   (both[:3], both[3:]), (both[:, :2], both[:, 2:])):
        with pytest.raises(Called):
            append(kp, vp)


def test_pages_of_any_order(lib):
    """Pages, rows and heads may lie in any order, with room between them; they may not lie over one another."""
    n = ctypes.c_size_t(0)

    def size(page, row, head, **kw):
        p = cache_params(page_stride=page, page_row_stride=row, page_head_stride=head, **kw)
        return lib.kda_cache_attention_workspace_size(ctypes.byref(p), ctypes.byref(n))
    N, P, HK, D = 20, 8, 2, 16
    for a, b, c in ((P * HK * D, HK * D, D), (P * HK * D, D, P * D), (HK * D, N * HK * D, D), (D, N * D, P * N * D),
                    (P * D, D, N * P * D), (D, HK * N * D, N * D), (1024, 2 * HK * D, D)):
        assert size(a, b, c) == OK, (a, b, c)
    for a, b, c in ((P * HK * D, 2 * HK * D, D), (P * HK * D, HK * D, 8), (HK * D, HK * D, D), (D, N * D, P * D), (D, D, D),
                    (P * HK * D - 8, HK * D, D)):
        assert size(a, b, c) == INVALID, (a, b, c)
    assert size(8, 8, 8, num_pages=1, page_size=1, num_kv_heads=1, num_q_heads=1) == OK       # extents of one
    assert size(1 << 40, 1 << 40, 1 << 40) == INVALID and size(1 << 40, D, 1 << 39) == OK
    for order in ("NPHD", "NHPD", "HNPD", "PNHD", "PHND", "HPND"):
        lens = dict(N=N, P=P, H=HK, D=D)
        x = torch.zeros([lens[c] for c in order]).permute([order.index(c) for c in "NPHD"])
        p = _lib.KdaCacheParams()
        cache._pages(p, x, x, torch.zeros(3, 2, dtype=torch.int32), 3)
        assert (p.page_stride, p.page_row_stride, p.page_head_stride) == x.stride()[:3]
    with pytest.raises(ValueError, match="overlap"):
        x = torch.zeros(9999).as_strided((N, P, HK, D), (P * HK * D, 2 * HK * D, D, 1))
        cache._pages(_lib.KdaCacheParams(), x, x, torch.zeros(3, 2, dtype=torch.int32), 3)
