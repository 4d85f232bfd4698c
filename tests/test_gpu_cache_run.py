"""The key-value cache's tables on the GPU against `oracle/cache.py`, and the operators together as a
hybrid model's server runs them: streams, captured graphs, forks beside the recurrent states."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
from gated_delta_rule_deltanet_gb300 import _lib, build as kbuild
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rng(*seed):
    return np.random.Generator(np.random.PCG64([*seed]))


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def no_error():
    torch.cuda.synchronize()
    assert kda.get_device_error() == 0


def page_error():
    torch.cuda.synchronize()
    with pytest.raises(Exception):
        if kda.get_device_error() == _lib.KDA_DEVERR_PAGE:
            raise RuntimeError
    assert kda.get_device_error() == 0


def random_tables(r, S, P, width, N, full=0.7):
    lens = r.integers(0, int(width * P * full) + 1, S)
    lens[r.random(S) < 0.15] = 0
    order = list(r.permutation(N))
    table, refs = np.full((S, width), -1, np.int32), np.zeros(N, np.int32)
    for s in range(S):
        for j in range(-(-lens[s] // P)):
            table[s, j] = order.pop()
            refs[table[s, j]] += 1
    return table, lens, refs


def check_update(table, lens, refs, parent, new, P, pools=(), **kw):
    ref = oc.update(table, lens, refs, parent if parent is not None else range(len(lens)), new, P)
    got = kda.cache_update(ints(table), ints(lens), ints(refs), None if parent is None else ints(parent), ints(new),
                           page_size=P, pools=pools, **kw)
    no_error()
    for name, x, y in zip(("table", "lens", "refs", "kept"), got, ref):
        assert np.array_equal(x.cpu().numpy(), y), name
    n = len(ref[4])
    pairs = np.stack([got.src.cpu().numpy(), got.dst.cpu().numpy()], 1)
    assert [tuple(x) for x in pairs[:n]] == ref[4] and np.all(pairs[n:] == -1)
    return got, ref


@pytest.mark.parametrize("S,P,width,N", [(1, 1, 1, 3), (3, 4, 5, 60), (40, 16, 9, 900), (300, 8, 33, 20000), (1100, 2, 7, 9000),
                                         (5000, 4, 3, 40000)])
def test_update_steps(S, P, width, N):
    """Random parents and lengths, step after step, so that pages come to be shared by many rows."""
    r = rng(1, S, P)
    table, lens, refs = random_tables(r, S, P, width, N)
    pool = torch.arange(N, device=DEV, dtype=torch.float32)[:, None].repeat(1, P).contiguous()
    for step in range(4 if S < 2000 else 2):
        parent = np.where(r.random(S) < 0.5, np.arange(S), r.integers(-1, S, S))
        new = np.where(parent >= 0, lens[np.maximum(parent, 0)] + r.integers(-3, 4, S), r.integers(0, 3 * P, S))
        new = np.clip(new, 0, width * P)
        before = pool.clone()
        got, ref = check_update(table, lens, refs, parent, new, P, pools=[pool])
        for a, b in ref[4]:
            before[b] = before[a]
        assert torch.equal(pool, before)
        table, lens, refs = ref[0], ref[1], ref[2]


def test_update_without_parents_and_with_another_number_of_rows():
    r = rng(2)
    table, lens, refs = random_tables(r, 20, 4, 8, 300)
    check_update(table, lens, refs, None, np.minimum(lens + 1, 32), 4)
    check_update(table, lens, refs, np.repeat(np.arange(20), 3), np.minimum(np.repeat(lens, 3) + 2, 32), 4)
    check_update(table, lens, refs, np.array([7, 7]), lens[[7, 7]], 4)
    check_update(table, lens, refs, np.full(5, -1), np.array([0, 1, 4, 5, 32]), 4)


@pytest.mark.parametrize("width", [64, 515, 516, 1100])
@pytest.mark.parametrize("shift", [0, 1])
def test_update_wide_tables(width, shift):
    """Rows of several rounds of a warp, by fours and one by one, of tables that begin anywhere."""
    r = rng(11, width)
    table, lens, refs = random_tables(r, 9, 2, width, 12000, full=0.9)
    parent, new = np.array([0, 0, 1, 5, 5, 5, -1, 8]), np.array([0] * 8)
    new = np.minimum(np.where(parent >= 0, lens[parent] + r.integers(-40, 40, 8), 777), 2 * width).clip(0)
    ref = oc.update(table, lens, refs, parent, new, 2)
    t = torch.full((9 * width + shift,), -7, dtype=torch.int32, device=DEV)[shift:].view(9, width)
    t.copy_(ints(table))
    o = [torch.empty(n + shift, dtype=torch.int32, device=DEV)[shift:] for n in (8 * width, 8, 12000, 8, 8, 8)]
    out = kda.CacheRows(o[0].view(8, width), *o[1:])
    kda.cache_update(t, ints(lens), ints(refs), ints(parent), ints(new), page_size=2, out=out)
    no_error()
    for x, y in zip(out, ref):
        if not isinstance(y, list):
            assert np.array_equal(x.cpu().numpy(), y)


def test_update_references_from_elsewhere():
    """A page that someone outside the table holds is copied before it is written, and stays when its rows end."""
    table, lens, refs = np.array([[0, 1], [2, -1]], np.int32), np.array([6, 3]), np.array([1, 2, 1, 0, 0, 0], np.int32)
    got, ref = check_update(table, lens, refs, None, np.array([7, 4]), 4)
    assert ref[4] == [(1, 3)] and ref[2][1] == 1
    got, ref = check_update(table, lens, refs, np.array([-1, -1]), np.array([0, 0]), 4)
    assert list(ref[2]) == [0, 1, 0, 0, 0, 0]


def test_update_pages_given_back_stay_so():
    table, lens = np.array([[-1, -1, 5, 1]], np.int32), np.array([15])
    refs = np.array([0, 1, 0, 0, 0, 1], np.int32)
    got, _ = check_update(table, lens, refs, None, np.array([16]), 4)
    got, _ = check_update(table, lens, refs, np.array([0, 0]), np.array([16, 14]), 4)
    assert got.table.cpu().tolist() == [[-1, -1, 5, 1], [-1, -1, 5, 0]]
    c = kda.cache_compact(ints(table), ints(lens), ints(refs), page_size=4)
    assert c.table.cpu().tolist() == [[-1, -1, 0, 1]]
    no_error()


@pytest.mark.parametrize("what", ["pages", "parent", "length", "negative", "entry", "free entry", "shared free entry", "refs", "old length"])
def test_update_refuses(what):
    """All or nothing: the new rows are empty, the counts as they were, nothing to copy."""
    table, lens = np.array([[0, 1], [2, 3]], np.int32), np.array([8, 5])
    refs, parent, new = np.array([1, 1, 1, 1, 0, 0], np.int32), np.array([0, 0, 1]), np.array([7, 6, 6])
    if what == "pages":
        parent, new = np.array([0, -1, -1]), np.array([8, 8, 4])
    elif what == "parent":
        parent[2] = 2
    elif what == "length":
        new[0] = 9
    elif what == "negative":
        new[1] = -1
    elif what == "entry":
        table[1, 0] = 6
    elif what == "free entry":
        refs[3] = 0
    elif what == "shared free entry":
        refs[0], parent = 0, np.array([0, 1, 1])
    elif what == "refs":
        refs[4] = -1
    else:
        lens[1] = 9
    got = kda.cache_update(ints(table), ints(lens), ints(refs), ints(parent), ints(new), page_size=4)
    page_error()
    assert torch.all(got.table == -1) and not got.lens.any() and not got.kept.any()
    assert torch.equal(got.refs, ints(refs)) and torch.all(got.src == -1) and torch.all(got.dst == -1)


def test_update_into_given_rows():
    r = rng(3)
    table, lens, refs = random_tables(r, 10, 4, 8, 200)
    out = kda.CacheRows(*(torch.full(s, 99, dtype=torch.int32, device=DEV)
                          for s in ((10, 8), (10,), (200,), (10,), (10,), (10,))))
    got, _ = check_update(table, lens, refs, None, np.minimum(lens + 3, 32), 4, out=out)
    assert got is out
    t = ints(table)
    with pytest.raises(ValueError, match="memory of its own"):
        kda.cache_update(t, ints(lens), ints(refs), None, ints(lens), page_size=4, out=out._replace(table=t))


@pytest.mark.parametrize("S,P,width,N", [(1, 1, 1, 1), (1, 4, 3, 2), (5, 4, 5, 61), (40, 16, 9, 1500), (300, 8, 33, 70001)])
def test_compact(S, P, width, N):
    r = rng(4, S, N)
    table, lens, refs = random_tables(r, S, P, width, N) if N > S * width else \
        (np.full((S, width), -1, np.int32), np.zeros(S, int), np.zeros(N, np.int32))
    if N > 10:
        refs[r.integers(0, N, 3)] += 1                       # pages that only others hold move, too
    pool = torch.from_numpy(r.standard_normal((N, P))).to(DEV, torch.bfloat16)
    before = pool.clone()
    got = kda.cache_compact(ints(table), ints(lens), ints(refs), page_size=P, pools=[pool])
    no_error()
    t, f, where, moves = oc.compact(table, lens, refs, P)
    assert np.array_equal(got.table.cpu(), t) and np.array_equal(got.refs.cpu(), f)
    assert np.array_equal(got.page_map.cpu(), where)
    pairs = np.stack([got.src.cpu().numpy(), got.dst.cpu().numpy()], 1) if N > 1 else np.zeros((0, 2))
    assert [tuple(x) for x in pairs[:len(moves)]] == moves and np.all(pairs[len(moves):] == -1)
    for a, b in moves:
        before[b] = before[a]
    assert torch.equal(pool, before)


def test_compact_full_and_empty_pools():
    table = np.array([[3, 1], [0, 2]], np.int32)
    got = kda.cache_compact(ints(table), ints([8, 7]), ints([1, 1, 1, 1]), page_size=4)
    assert torch.equal(got.table, ints(table)) and torch.all(got.src == -1)
    got = kda.cache_compact(ints(table), ints([0, 0]), ints([0, 0, 0, 0]), page_size=4)
    assert torch.all(got.table == -1) and torch.all(got.page_map == -1)
    no_error()


@pytest.mark.parametrize("what", ["free", "range", "refs", "length"])
def test_compact_refuses(what):
    table, lens, refs = np.array([[5, 3]], np.int32), np.array([8]), np.array([0, 0, 0, 1, 0, 1], np.int32)
    if what == "free":
        refs[3] = 0
    elif what == "range":
        table[0, 0] = 6
    elif what == "refs":
        refs[0] = -2
    else:
        lens[0] = 9
    got = kda.cache_compact(ints(table), ints(lens), ints(refs), page_size=4)
    page_error()
    assert torch.equal(got.table, ints(table)) and torch.equal(got.refs, ints(refs)) and torch.all(got.src == -1)


@pytest.mark.parametrize("shapes", [[(9, 4, 2, 16)], [(9, 4, 2, 16), (9, 4, 2, 16), (9, 3)], [(9, 5000)], [(9, 7)], [(9,)],
                                    [(9, 33)] * 70])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8])
def test_copy(shapes, dtype):
    """Pools of any type and size, more of them than one launch takes; the list ends at its first negative source."""
    pools = [torch.randint(0, 100, s, device=DEV).to(dtype) for s in shapes]
    want = [p.clone() for p in pools]
    src, dst = [4, 8, 4, -1, -1], [0, 7, 3, -1, -1]
    for w in want:
        for a, b in zip(src[:3], dst[:3]):
            w[b] = w[a]
    kda.cache_copy(pools, ints(src), ints(dst))
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    kda.cache_copy(pools, ints([]), ints([]))
    no_error()


def test_copy_strided_pages_and_bad_indices():
    whole = torch.randn((6, 2, 40), device=DEV)
    want = whole.clone()
    want[1, 0] = want[5, 0]
    kda.cache_copy([whole[:, 0]], ints([5]), ints([1]))      # the other half of each page stays
    assert torch.equal(whole, want)
    no_error()
    kda.cache_copy([whole], ints([6, 2, 3]), ints([0, 9, 4]))
    page_error()
    want[4] = want[3]
    assert torch.equal(whole, want)


# ---------------------------------------------------------------------------------------- together

class Server:
    """A layer of attention beside a layer of the recurrence: rows of both for S sequences."""

    def __init__(self, S=6, P=16, N=120, H=4, HK=2, D=64, dtype=torch.bfloat16):
        self.S, self.P, self.N, self.H, self.HK, self.D = S, P, N, H, HK, D
        z = dict(device=DEV)
        self.k_pages, self.v_pages = (torch.zeros((N, P, HK, D), dtype=dtype, **z) for _ in range(2))
        self.rows = kda.CacheRows(torch.full((S, 20), -1, dtype=torch.int32, **z), ints([0] * S), ints([0] * N),
                                  ints([0] * S), ints([-1] * S), ints([-1] * S))
        self.freq, _ = kda.rotary_frequencies(D, device=DEV)
        self.state = torch.zeros((S, 2, 16, 16), **z)

    def step(self, parent, grow, q, k, v, offsets=None, window=1):
        r = self.rows
        lens = r.lens[parent.clamp(min=0)] * (parent >= 0)
        self.rows = kda.cache_update(r.table, r.lens, r.refs, parent, (lens + grow).to(torch.int32), page_size=self.P,
                                     pools=[self.k_pages, self.v_pages])
        qr = kda.cache_append(q, k, v, self.freq, self.k_pages, self.v_pages, self.rows.table, self.rows.kept,
                              input_row_offsets=offsets)
        return kda.cache_attention(qr, self.k_pages, self.v_pages, self.rows.table, self.rows.lens, window=window)


def replay(hist, freq, H, HK, D):
    """fp64 attention of the last token of a history of (q, k, v)."""
    n = len(hist)
    q, k, v = (np.stack([h[i] for h in hist]) for i in range(3))
    k = oc.rotary(k, range(n), freq)
    q = oc.rotary(q[-1:], [n - 1], freq)
    return oc.attention(q, k, v, 1, D ** -0.5)[0][0]


def test_a_server_of_a_hybrid_model():
    """Prompts in windows, decoding, forks, cut-back drafts, sequences that end and begin, a compaction: every token's
    output is that of its own history.  A token's rotated q and k are rounded to bf16 once (2^-8 of values of
    size ~4 at most), which moves scores by up to 2 * 2^-8 * sum|q k| / sqrt(D) ~ 0.05 and o by as much of values of size ~1."""
    r = rng(5)
    s = Server()
    S, H, HK, D = s.S, s.H, s.HK, s.D
    freq = s.freq.cpu().numpy()
    hist = [[] for _ in range(S)]

    def fresh(n):
        t = [torch.from_numpy(r.standard_normal((n, h, D)).astype(np.float32)).to(DEV, torch.bfloat16) for h in (H, HK, HK)]
        return t, [x.double().cpu().numpy() for x in t]

    def run(parent, grow, window=1, keep=None):
        nonlocal hist
        grow = np.broadcast_to(grow, (S,))
        (q, k, v), (q64, k64, v64) = fresh(int(grow.sum()))
        offsets = np.concatenate([[0], np.cumsum(grow)])
        o = s.step(ints(parent), ints(grow), q, k, v, ints(offsets), window)
        new = []
        for i, p in enumerate(parent):
            h = list(hist[p]) if p >= 0 else []
            for j in range(grow[i]):
                h.append((q64[offsets[i] + j], k64[offsets[i] + j], v64[offsets[i] + j]))
                if window == 1 or grow[i] == window:
                    if window > 1 or j == grow[i] - 1:
                        got = o[i * window + (j if window > 1 else 0)].double().cpu().numpy()
                        assert np.max(np.abs(got - replay(h, freq, H, HK, D))) < 0.06
            new.append(h)
        hist = new
        assert [len(h) for h in hist] == s.rows.lens.cpu().tolist()

    everyone = list(range(S))
    run([-1] * S, 13, window=13)                             # prompts, all of a window
    for _ in range(4):
        run(everyone, 1)
    run([0, 0, 0, 3, 3, 5], 1)                               # forks; rows 1, 2 and 4 end
    for _ in range(3):
        run(everyone, 1)
    # a draft window of four, of which two are taken
    run(everyone, 4, window=4)
    r_ = s.rows
    s.rows = kda.cache_update(r_.table, r_.lens, r_.refs, None, r_.lens - 2, page_size=s.P, pools=[s.k_pages, s.v_pages])
    hist = [h[:-2] for h in hist]
    run(everyone, 1)
    run([0, -1, 2, 2, -1, 5], [1, 1, 1, 1, 1, 1])            # two sequences end, two begin
    m = kda.cache_compact(s.rows.table, s.rows.lens, s.rows.refs, page_size=s.P, pools=[s.k_pages, s.v_pages])
    used = int((m.refs > 0).sum())
    assert not m.refs[used:].any()
    s.k_pages[used:] = float("nan")
    s.v_pages[used:] = float("nan")
    s.rows = s.rows._replace(table=m.table, refs=m.refs)
    run(everyone, 1)
    assert torch.equal(s.rows.refs, torch.bincount(s.rows.table[s.rows.table >= 0].long(), minlength=s.N).int())
    no_error()


def test_forked_sequences_keep_their_recurrent_state():
    """cache_copy on a state pool: the fork's decode steps are its parent's."""
    r = rng(6)
    pool = torch.from_numpy(r.standard_normal((8, 2, 16, 16)).astype(np.float32)).to(DEV)
    conv = torch.from_numpy(r.standard_normal((8, 96, 3)).astype(np.float32)).to(DEV)
    kda.cache_copy([pool], ints([1, 1, -1]), ints([4, 6, -1]))
    kda.cache_copy([conv], ints([1, 1, -1]), ints([4, 6, -1]))
    assert torch.equal(conv[4], conv[1]) and torch.equal(conv[6], conv[1])
    q, k, v = (torch.from_numpy(r.standard_normal((1, 2, 16)).astype(np.float32)).to(DEV).repeat(3, 1, 1) for _ in range(3))
    beta, g = torch.full((3, 2), 0.5, device=DEV), torch.full((3, 2), -0.1, device=DEV)
    o = kda.decode_step(q, k, v, beta, g, ints([1, 4, 6]), pool)
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2]) and torch.equal(pool[1], pool[6])
    no_error()


def test_streams():
    """The whole chain on a stream that is not the current one, its inputs made there."""
    st = torch.cuda.Stream()
    r = rng(7)
    x = torch.from_numpy(r.standard_normal((2, 4, 64)).astype(np.float32)).to(DEV, torch.bfloat16)
    pages = torch.zeros((8, 16, 4, 64), dtype=torch.bfloat16, device=DEV)
    f, _ = kda.rotary_frequencies(64, device=DEV)
    a = [pages.clone(), pages.clone()]
    table, zero = ints([[2], [5]]), ints([0, 0])
    want = kda.cache_attention(kda.cache_append(x, x, x, f, a[0], a[1], table, zero), a[0], a[1], table, ints([1, 1]))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(10000000)                          # the call has to wait for what its own stream makes
        b = [pages.clone(), pages.clone()]
        y = x + 0
    q = kda.cache_append(y, y, y, f, b[0], b[1], table, zero, stream=st)
    o = kda.cache_attention(q, b[0], b[1], table, ints([1, 1]), stream=st)
    t, _ = kda.rotary(y, None, ints([0, 0]), f, stream=st)
    kda.cache_copy(b, ints([2]), ints([0]), stream=st)
    u = kda.cache_update(table, ints([1, 1]), ints([0, 0, 1, 0, 0, 1, 0, 0]), None, ints([2, 2]), page_size=16, stream=st)
    st.synchronize()
    assert torch.equal(o, want) and torch.equal(b[0][0], b[0][2]) and torch.equal(u.table, table) and torch.equal(t, x)
    no_error()


def test_two_calls_at_once_do_not_share():
    """Splits on two streams at the same time, each with a workspace of its own."""
    r = rng(8)
    kp = torch.from_numpy(r.standard_normal((600, 16, 2, 64)).astype(np.float32)).to(DEV, torch.bfloat16)
    table = ints(np.arange(600)[None])
    qs = [torch.from_numpy(r.standard_normal((1, 4, 64)).astype(np.float32)).to(DEV, torch.bfloat16) for _ in range(2)]
    want = [kda.cache_attention(q, kp, kp, table, ints([9600 - 7 * i])) for i, q in enumerate(qs)]
    lens = [ints([9600 - 7 * i]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [kda.cache_attention(q, kp, kp, table, n, stream=s) for q, n, s in zip(qs, lens, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_captured_decode_step_follows_its_inputs():
    """Update, append and attention in one graph, the tables going from one buffer to the other and back: lengths,
    parents and tokens change between replays."""
    r = rng(9)
    S, P, N, HK, D = 5, 4, 60, 2, 32
    kp, vp = (torch.zeros((N, P, HK, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    f, _ = kda.rotary_frequencies(D, device=DEV)
    z = dict(dtype=torch.int32, device=DEV)
    bufs = [kda.CacheRows(torch.full((S, 8), -1, **z), torch.zeros(S, **z), torch.zeros(N, **z), torch.zeros(S, **z),
                          torch.full((S,), -1, **z), torch.full((S,), -1, **z)) for _ in range(2)]
    x = torch.zeros((S, HK, D), dtype=torch.bfloat16, device=DEV)
    parent, new = ints([-1] * S), ints([1] * S)

    def step(a, b):
        kda.cache_update(a.table, a.lens, a.refs, parent, new, page_size=P, pools=[kp, vp], out=b)
        q = kda.cache_append(x, x, x, f, kp, vp, b.table, b.kept)
        return kda.cache_attention(q, kp, vp, b.table, b.lens)

    step(bufs[0], bufs[1])                                   # the first calls of the process outside the capture
    kp.zero_()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(bufs[i], bufs[1 - i]))
        graphs.append(g)
    hist = [[] for _ in range(S)]
    bufs[0].lens.zero_()
    bufs[0].refs.zero_()
    for t in range(9):
        p = [-1] * S if t == 0 else list(range(S)) if t % 3 else [0, 0, 2, 2, 4]
        y = torch.from_numpy(r.standard_normal((S, HK, D)).astype(np.float32)).to(torch.bfloat16)
        x.copy_(y)
        y = y.double().numpy()
        hist = [(list(hist[q]) if q >= 0 else []) + [(y[i], y[i], y[i])] for i, q in enumerate(p)]
        parent.copy_(ints(p))
        new.copy_(ints([len(h) for h in hist]))
        graphs[t % 2].replay()
        got = outs[t % 2].double().cpu().numpy()
        for i in range(S):
            # as in test_a_server_of_a_hybrid_model
            assert np.max(np.abs(got[i] - replay(hist[i], f.cpu().numpy(), HK, HK, D))) < 0.06
    no_error()


def test_workspaces_of_the_caller():
    r = rng(10)
    kp = torch.from_numpy(r.standard_normal((40, 16, 1, 32)).astype(np.float32)).to(DEV, torch.bfloat16)
    q = torch.from_numpy(r.standard_normal((1, 2, 32)).astype(np.float32)).to(DEV, torch.bfloat16)
    table = ints(np.arange(40)[None])
    want = kda.cache_attention(q, kp, kp, table, ints([600]))
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device=DEV)
    assert torch.equal(kda.cache_attention(q, kp, kp, table, ints([600]), workspace=ws), want)
    a = kda.cache_update(table, ints([600]), ints([1] * 38 + [0, 0]), None, ints([608]), page_size=16)
    b = kda.cache_update(table, ints([600]), ints([1] * 38 + [0, 0]), None, ints([608]), page_size=16, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(ValueError, match="bytes"):
        kda.cache_attention(q, kp, kp, table, ints([600]), workspace=ws[:1024])
    no_error()


def test_an_attention_sublayer_is_trained_through_its_rotation():
    """rotary and rotary_bwd as an autograd pair around an eager attention: gradients of q and k as autograd forms them
    through the written-out rotation."""
    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, pos, f):
            ctx.save_for_backward(pos, f)
            return kda.rotary(q, k, pos, f)

        @staticmethod
        def backward(ctx, dq, dk):
            return (*kda.rotary_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors), None, None)

    T, H, D = 12, 2, 16
    f, _ = kda.rotary_frequencies(D, device=DEV)
    pos = torch.arange(T, device=DEV)
    leaves = [torch.randn((T, H, D), device=DEV, requires_grad=True) for _ in range(2)]

    def plain(x):
        a, b = x[..., :D // 2], x[..., D // 2:]
        ang = (pos[:, None] * f)[:, None]
        c, s = ang.cos().float(), ang.sin().float()
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    grads = []
    for turn in (lambda q, k: Turn.apply(q, k, pos, f), lambda q, k: (plain(q), plain(k))):
        q, k = turn(*leaves)
        torch.softmax(torch.einsum("thd,shd->hts", q, k), -1).square().sum().backward()
        grads.append([x.grad.clone() for x in leaves])
        for x in leaves:
            x.grad = None
    for a, b in zip(*grads):
        # both in fp32 through a softmax of sums of 16 products: a few hundred roundings of terms up to |q| |k| ~ 40
        assert torch.allclose(a, b, rtol=1e-4, atol=1e-4)


def test_tables_of_nothing():
    z = dict(dtype=torch.int32, device=DEV)
    r = kda.cache_update(torch.empty((0, 4), **z), ints([]), ints([0, 0, 2]), ints([-1, -1]), ints([3, 0]), page_size=2)
    assert r.table.cpu().tolist() == [[0, 1, -1, -1], [-1] * 4] and r.refs.cpu().tolist() == [1, 1, 2]
    r = kda.cache_update(torch.empty((0, 4), **z), ints([]), ints([]), None, ints([]), page_size=2)
    assert r.table.shape == (0, 4)
    r = kda.cache_update(ints([[1]]), ints([2]), ints([0, 1]), ints([]), ints([]), page_size=2)       # every row ends
    assert r.refs.cpu().tolist() == [0, 0]
    c = kda.cache_compact(torch.empty((0, 4), **z), ints([]), ints([0, 3, 0]), page_size=2)
    assert c.page_map.cpu().tolist() == [-1, 0, -1]
    c = kda.cache_compact(torch.full((2, 1), -1, **z), ints([0, 0]), ints([]), page_size=2)
    assert torch.all(c.table == -1)
    no_error()


def test_update_asks_for_more_pages_than_there_are_in_all():
    """Needs whose sum passes 2^31."""
    S, width = 40000, 60000
    table = torch.empty((0, width), dtype=torch.int32, device=DEV)
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    r = kda.cache_update(table, ints([]), ints([0] * 50), ints([-1] * S), ints([width] * S), page_size=1)
    page_error()
    assert not r.lens.any() and not r.refs.any()


FIRST_CALLS = """
import torch
import gated_delta_rule_deltanet_gb300 as kda
dev = "cuda:0"
f = torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64, device=dev)
x = torch.randn((3, 2, 64), device=dev).bfloat16()
y = torch.randn((3, 2, 32), device=dev)
pages = [torch.randn((9, 4, 2, 64), device=dev).bfloat16() for _ in range(2)]
wide = [torch.randn((9, 4, 2, 32), device=dev) for _ in range(2)]
i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
table, lens, refs = torch.tensor([[0, 1], [2, -1], [3, -1]], dtype=torch.int32, device=dev), i(5, 1, 4), i(1, 1, 1, 1, 0, 0, 0, 0, 0)
parent, new, start = i(0, 0, 2), i(6, 6, 5), i(4, 0, 3)

def calls():
    a = kda.cache_append(x, x, x, f, *pages, table, start)
    return [a, *kda.rotary(x, x, start, f), kda.cache_attention(a, *pages, table, lens),
            kda.cache_attention(y, *wide, table, lens),
            *kda.cache_update(table, lens, refs, parent, new, page_size=4, pools=pages),
            *kda.cache_compact(table, lens, refs, page_size=4, pools=wide)]

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = calls()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, calls())) and kda.get_device_error() == 0
"""


def test_first_calls_of_a_process_may_be_captured():
    subprocess.run([sys.executable, "-c", FIRST_CALLS], check=True, cwd=kbuild.ROOT, timeout=300)
