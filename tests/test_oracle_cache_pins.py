"""The fp64 reference of the key-value cache against facts that do not restate its formulas."""
import numpy as np
import pytest

from oracle import cache as oc


def rng(*seed):
    return np.random.Generator(np.random.PCG64([*seed]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_scores_depend_on_the_distance_alone(interleaved):
    r = rng(1, interleaved)
    q, k = r.standard_normal((1, 1, 12)), r.standard_normal((1, 1, 12))
    f, _ = oc.frequencies(12)
    at = [(oc.rotary(q, [p], f, interleaved) * oc.rotary(k, [p - 7], f, interleaved)).sum() for p in (7, 50, 1000)]
    assert np.allclose(at, at[0], atol=1e-12)


def test_rotary_of_position_zero_and_its_length():
    x = rng(2).standard_normal((3, 2, 10))
    f, _ = oc.frequencies(6)
    assert np.array_equal(oc.rotary(x, [0, 0, 0], f), x)
    y = oc.rotary(x, [5, -3, 12345], f, magnitude=1.5)
    assert np.allclose((y[..., :6] ** 2).sum(-1), 2.25 * (x[..., :6] ** 2).sum(-1))
    assert np.array_equal(y[..., 6:], x[..., 6:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient_by_differences(interleaved):
    r = rng(3, interleaved)
    x, d = r.standard_normal((2, 1, 8)), r.standard_normal((2, 1, 8))
    f, _ = oc.frequencies(6)
    pos = [11, 300]
    g = oc.rotary(d, pos, f, interleaved, 1.2, transpose=True)
    g[..., 6:] = d[..., 6:]                    # the channels that pass
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        diff = ((oc.rotary(x + e, pos, f, interleaved, 1.2) - oc.rotary(x - e, pos, f, interleaved, 1.2)) * d).sum() / (2 * h)
        assert abs(diff - g[i]) < 1e-8


def test_frequency_scalings():
    plain, _ = oc.frequencies(16)
    assert np.allclose(oc.frequencies(16, scaling="linear", factor=4)[0], plain / 4)
    ntk = oc.frequencies(16, scaling="ntk", factor=4)[0]
    assert np.isclose(ntk[0], plain[0]) and np.isclose(ntk[-1], plain[-1] / 4)
    parts, m = oc.frequencies(64, scaling="by_parts", factor=8, trained_length=4096)
    ratio = parts / oc.frequencies(64)[0]
    assert np.isclose(ratio[0], 1) and np.isclose(ratio[-1], 1 / 8) and np.all(np.diff(ratio) <= 1e-15)
    assert np.isclose(m, 1 + 0.1 * np.log(8))


def test_attention_of_equal_keys_is_the_mean():
    v = rng(4).standard_normal((9, 1, 5))
    k = np.ones((9, 1, 5))
    o, lse, *_ = oc.attention(np.ones((1, 2, 5)), k, v, 1, 0.3)
    assert np.allclose(o, v.mean(0)) and np.allclose(lse, 1.5 + np.log(9))


def test_attention_span_window_and_slopes():
    r = rng(5)
    q, k, v = r.standard_normal((3, 2, 4)), r.standard_normal((8, 1, 4)), r.standard_normal((8, 1, 4))
    o, lse, *_ = oc.attention(q, k, v, 3, 0.5, span=1)
    assert np.allclose(o, v[5:].repeat(2, 1))                 # a query that sees itself alone
    a, la, *_ = oc.attention(q[:1], k[:6], v[:6], 1, 0.5)     # a window's first query sees no later key
    b, lb, *_ = oc.attention(q, k, v, 3, 0.5)
    assert np.allclose(a[0], b[0]) and np.allclose(la[0], lb[0])
    far, *_ = oc.attention(q, k, v, 3, 0.5, slopes=np.array([1e4, 1e4]))
    assert np.allclose(far, v[5:].repeat(2, 1))               # a steep slope leaves the nearest key
    e, le, *_ = oc.attention(q, k[:0], v[:0], 3, 0.5)
    assert not e.any() and np.all(le == -np.inf)


def test_attention_parts_join_by_their_lse():
    r = rng(6)
    q, k, v = r.standard_normal((1, 1, 4)), r.standard_normal((20, 1, 4)), r.standard_normal((20, 1, 4))
    o, lse, *_ = oc.attention(q, k, v, 1, 1.0, softcap=2.0)
    parts = [oc.attention(q, k[a:b], v[a:b], 1, 1.0, softcap=2.0) for a, b in ((0, 7), (7, 20))]
    w = [np.exp(p[1] - lse)[..., None] for p in parts]
    assert np.allclose(sum(x * p[0] for x, p in zip(w, parts)), o)


def random_cache(r, S, P, width, N):
    lens = r.integers(0, width * P + 1, S)
    lens[r.random(S) < 0.2] = 0
    order = list(r.permutation(N))
    table, refs = np.full((S, width), -1, np.int32), np.zeros(N, np.int32)
    for s in range(S):
        for j in range(-(-lens[s] // P)):
            table[s, j] = order.pop()
            refs[table[s, j]] += 1
    return table, lens, refs


@pytest.mark.parametrize("seed", range(6))
def test_update_keeps_every_rows_tokens_and_owns_what_is_written(seed):
    r = rng(7, seed)
    S, P, width, N = 7, 4, 6, 400
    table, lens, refs = random_cache(r, S, P, width, N)
    content = r.permutation(N * P).reshape(N, P)
    for _ in range(4):                                        # steps one after another: pages come to be shared
        parent = r.integers(-1, S, S)
        new = r.integers(0, width * P + 1, S)
        t, n, f, kept, copies = oc.update(table, lens, refs, parent, new, P)
        after = content.copy()
        for a, b in copies:
            assert refs[b] == 0                               # the old tables stay valid
            after[b] = content[a]
        for i, p in enumerate(parent):
            for j in range(kept[i]):
                assert after[t[i, j // P], j % P] == content[table[p, j // P], j % P]
            for j in range(kept[i], new[i]):                  # what will be written belongs to one row
                assert f[t[i, j // P]] == 1 and (t == t[i, j // P]).sum() == 1
        assert np.array_equal(f, np.bincount(t[t >= 0], minlength=N))
        table, lens, refs, content = t, n, f, after


def test_compact_moves_as_few_pages_as_can_be():
    r = rng(8)
    table, lens, refs = random_cache(r, 6, 4, 5, 60)
    t, f, where, moves = oc.compact(table, lens, refs, 4)
    n = (refs > 0).sum()
    assert np.all(f[:n] > 0) and not f[n:].any() and len(moves) == (refs[n:] > 0).sum()
    assert all(refs[b] == 0 for _, b in moves)
    assert np.array_equal(np.where(table >= 0, where[table], -1), t)


@pytest.mark.parametrize("parent", [[0, 1], [1, 1], [0, 0], [-1, -1]])
@pytest.mark.parametrize("page", range(4))
def test_update_takes_no_row_that_names_a_free_page(parent, page):
    table, refs = np.array([[0, 1], [2, 3]], np.int32), np.array([1, 1, 1, 1, 0, 0, 0, 0], np.int32)
    oc.update(table, [8, 5], refs, parent, [8, 8], 4)
    refs[page] = 0
    with pytest.raises(ValueError, match="free page"):
        oc.update(table, [8, 5], refs, parent, [8, 8], 4)
