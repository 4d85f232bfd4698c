"""Torch-facing binding of the key-value cache of a hybrid model's attention layers: rotary positions,
the pages that keys and values are written to, attention of new tokens over them, and the page
tables (kda_rotary_*, kda_cache_*).  Argument marshalling only, as in `layer.py`.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Sequence

import torch

from . import _lib
from ._lib import KdaCacheParams, KdaCacheRowsParams, KdaError, KdaRotaryParams
from .kda import _INDEX_DTYPES, _QKV_DTYPES
from .layer import (_PLANS, _Plan, _apart, _call, _current_device, _dense, _device, _keep, _on, _p, _pairs,
                    _raw_stream, _sig, _sig16, _space)

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = ("none", "linear", "ntk", "by_parts")


# ---------------------------------------------------------------------------------------- positions

def rotary_frequencies(rot_dim: int, *, base: float = 10000.0, scaling: str = "none",
                       factor: float = 1.0, trained_length: int = 0, slow: float = 1.0,
                       fast: float = 32.0, device="cuda"):
    """Frequencies of the pairs of `rot_dim` turned channels, base^(-2 i / rot_dim) radians per
    position, and the factor of the turned values: what `rotary` and `cache_append` take.

    For contexts `factor` times as long as trained: `linear` divides every frequency (Chen et al.,
    "Extending context window of large language models via positional interpolation", 2023); `ntk`
    raises the base so that the slowest pair's is divided and the fastest's kept; `by_parts` divides
    those of pairs that turn less than `slow` times over `trained_length` positions, keeps those that turn more than
    `fast` times and blends between, with the factor 0.1 ln(factor) + 1 (Peng et al., "YaRN", 2023).
    Returns (float64 [rot_dim / 2] on `device`, magnitude)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2 * i / rot_dim) for i in range(rot_dim // 2)]
    magnitude = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "by_parts":
        if trained_length < 1 or not fast > slow:
            raise ValueError("by_parts needs trained_length and fast > slow")
        keep = [min(1.0, max(0.0, (trained_length * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
        magnitude = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    return torch.tensor(f, dtype=torch.float64, device=device), magnitude


def _heads(t, name, like=None):
    """[T, H, d] with dense heads and any row stride; returns the elements between rows."""
    if t.dim() != 3 or t.dtype not in _QKV_DTYPES:
        raise ValueError(f"{name} must be [T, H, d] float32 or bfloat16")
    if like is not None and (t.dtype != like.dtype or t.shape[0] != like.shape[0] or t.shape[2] != like.shape[2]):
        raise ValueError(f"{name} must have the dtype, tokens and head size of the other heads")
    T, H, D = t.shape
    if H * D and ((D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D)):
        raise ValueError(f"{name} must have dense (H, d) rows")
    if T > 1 and H * D:
        if t.stride(0) < H * D:
            raise ValueError(f"{name}'s rows must not overlap")
        return t.stride(0)
    return 0


def _layout(layout):
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {', '.join(_LAYOUTS)}")
    return _LAYOUTS[layout]


def _frequencies(f, D):
    if f is None:
        return 0
    if f.dim() != 1 or f.dtype != torch.float64 or not f.is_contiguous() or f.numel() < 1 or 2 * f.numel() > D:
        raise ValueError("frequencies must be contiguous float64 [R / 2], R at most the head size")
    return 2 * f.numel()


def _place(out, x, name):
    """Checks an output that is given."""
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{name} must be shaped and typed like its input")
    return _heads(out, name)


def _plan_rotary(key, name, q, k, positions, frequencies, layout, magnitude, q_out, k_out):
    dev = _device(q, k, positions, frequencies, q_out, k_out)
    p = KdaRotaryParams(tokens=q.shape[0], num_q_heads=q.shape[1], head_dim=q.shape[2], q_row_stride=_heads(q, "q"),
                        dtype=_QKV_DTYPES[q.dtype], interleaved=_layout(layout), magnitude=magnitude,
                        rot_dim=_frequencies(frequencies, q.shape[2]))
    if k is not None:
        p.k_row_stride = _heads(k, "k", q)
        p.num_k_heads = k.shape[1]
    if positions.shape != (q.shape[0],) or positions.dtype not in (torch.int32, torch.int64) \
            or not positions.is_contiguous():
        raise ValueError("positions must be contiguous int32 or int64 [T]")
    p.wide_positions = positions.dtype == torch.int64
    if q_out is not None:
        p.q_out_row_stride = _place(q_out, q, "q_out")
    if k_out is not None:
        if k is None:
            raise ValueError("k_out needs k")
        p.k_out_row_stride = _place(k_out, k, "k_out")
    return _keep(key, _Plan(name, p, dev))


def _rotary(name, q, k, positions, frequencies, layout, magnitude, q_out, k_out):
    magnitude = float(magnitude)
    key = (name, _sig(q), _sig(k), _sig(positions), _sig(frequencies), layout, magnitude, _sig(q_out), _sig(k_out))
    plan = _PLANS.get(key)
    if plan is None:
        pairs = _apart(_pairs((q, k, q_out, k_out), ("q_out", 2, 0, True), ("q_out", 2, 1), ("q_out", 2, 3),
                              ("k_out", 3, 0), ("k_out", 3, 1, True)), q, k, q_out, k_out)
        if frequencies is None:
            raise ValueError("frequencies must be contiguous float64 [R / 2], R at most the head size")
        plan = _plan_rotary(key, name, q, k, positions, frequencies, layout, magnitude, q_out, k_out)
        plan.pairs = pairs
    elif plan.pairs:
        _apart(plan.pairs, q, k, q_out, k_out)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=plan.device)
    if k_out is None and k is not None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=plan.device)
    _call(plan, q.data_ptr(), _p(k), positions.data_ptr(), frequencies.data_ptr(), q_out.data_ptr(), _p(k_out))
    return q_out, k_out


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
           frequencies: torch.Tensor, *, layout: str = "half", magnitude: float = 1.0,
           q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
           stream: Optional[torch.cuda.Stream] = None):
    """Rotary positions (kda_rotary_fwd): the channel pairs of q [T, H, d] and k [T, HK, d] (or None)
    turned by positions[t] * frequencies[i] and multiplied by `magnitude`; channels from
    2 * frequencies.numel() on pass.  `layout`: pairs (i, i + R/2) ("half") or (2i, 2i + 1)
    ("interleaved").  positions [T] int32 or int64: angles are formed in 64-bit fixed point, off
    by up to 2^-28 + |p f| 2^-55 of a turn (2^-24 at 2^31 and one radian a position); frequencies as `rotary_frequencies`
    returns them.  q and k may be column blocks of a packed projection.
    Returns (q', k'), dense unless `q_out` / `k_out` are given, which may be q and k themselves."""
    if stream is not None:
        with _on(stream, q):
            return rotary(q, k, positions, frequencies, layout=layout, magnitude=magnitude, q_out=q_out, k_out=k_out)
    return _rotary("kda_rotary_fwd", q, k, positions, frequencies, layout, magnitude, q_out, k_out)


def rotary_bwd(d_q: torch.Tensor, d_k: Optional[torch.Tensor], positions: torch.Tensor,
               frequencies: torch.Tensor, *, layout: str = "half", magnitude: float = 1.0,
               dq_out: Optional[torch.Tensor] = None, dk_out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """Backward of `rotary` (kda_rotary_bwd): the gradients of q and k from those of the turned ones.
    Arguments as there."""
    if stream is not None:
        with _on(stream, d_q):
            return rotary_bwd(d_q, d_k, positions, frequencies, layout=layout, magnitude=magnitude, dq_out=dq_out,
                              dk_out=dk_out)
    return _rotary("kda_rotary_bwd", d_q, d_k, positions, frequencies, layout, magnitude, dq_out, dk_out)


# -------------------------------------------------------------------------------------------- pages

def _pages(p, k_pages, v_pages, block_table, B):
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or k_pages.dtype not in _QKV_DTYPES \
            or v_pages.dtype != k_pages.dtype or v_pages.stride() != k_pages.stride():
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, HK, d] of one dtype and stride")
    N, P, HK, D = k_pages.shape
    if P < 1 or HK < 1 or D < 1 or (D > 1 and k_pages.stride(3) != 1):
        raise ValueError("the pages' heads must be dense")
    # strides of extents of one say nothing; the library takes those of dense pages there
    head = k_pages.stride(2) if HK > 1 else D
    row = k_pages.stride(1) if P > 1 else HK * D
    page = k_pages.stride(0) if N > 1 else P * HK * D
    span = D
    for apart, n in sorted(((head, HK), (row, P), (page, N))):
        if n > 1 and apart < span:
            raise ValueError("the pages' heads must not overlap")
        span += apart * max(0, n - 1)
    if block_table.dim() != 2 or block_table.shape[0] != B or block_table.dtype != torch.int32 \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [num_seqs, max_pages]")
    p.num_seqs, p.num_kv_heads, p.head_dim, p.page_size, p.num_pages = B, HK, D, P, N
    p.max_pages = block_table.shape[1]
    p.dtype = _QKV_DTYPES[k_pages.dtype]
    p.page_stride, p.page_row_stride, p.page_head_stride = page, row, head


def _index(t, n, name):
    if t.shape != (n,) or t.dtype not in _INDEX_DTYPES or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [{n}]")


def _plan_append(key, q, k, v, frequencies, k_pages, v_pages, block_table, start, offsets, layout, magnitude, q_out):
    dev = _device(q, k, v, frequencies, k_pages, v_pages, block_table, start, offsets, q_out)
    p = KdaCacheParams(tokens=k.shape[0], interleaved=_layout(layout), magnitude=magnitude, o_dtype=0)
    B = start.numel()
    _pages(p, k_pages, v_pages, block_table, B)
    _index(start, B, "start")
    if k.shape != (k.shape[0], p.num_kv_heads, p.head_dim) or v.shape != k.shape or k.dtype != k_pages.dtype:
        raise ValueError("k and v must be [T, HK, d] in the pages' dtype")
    p.k_row_stride, p.v_row_stride = _heads(k, "k"), _heads(v, "v", k)
    p.rot_dim = _frequencies(frequencies, p.head_dim)
    if q is not None:
        p.q_row_stride = _heads(q, "q", k)
        p.num_q_heads = q.shape[1]
        if q_out is not None:
            p.q_out_row_stride = _place(q_out, q, "q_out")
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if offsets is None:
        if p.tokens != B:
            raise ValueError("without input_row_offsets each token is a sequence: start must be [T]")
    else:
        _index(offsets, B + 1, "input_row_offsets")
    return _keep(key, _Plan("kda_cache_append", p, dev))


def cache_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
                 frequencies: Optional[torch.Tensor], k_pages: torch.Tensor, v_pages: torch.Tensor,
                 block_table: torch.Tensor, start: torch.Tensor, *,
                 input_row_offsets: Optional[torch.Tensor] = None, layout: str = "half",
                 magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """New tokens into the cache (kda_cache_append): k [T, HK, d] turned as in `rotary` and v written
    into the pages, q [T, H, d] (or None) turned and returned.

    k_pages, v_pages [num_pages, page_size, HK, d], any strides that keep the heads' channels together
    (permuted views of [num_pages, HK, page_size, d], [HK, num_pages, page_size, d] and the like too), that
    share no memory; block_table [B, max_pages] int32; start [B] int32: the tokens that each sequence
    already holds, the position of its first new one.
    Without `input_row_offsets` every row is a sequence's one new token (the decode form); with it, tokens from
    its last entry on are left alone.  `frequencies` None: nothing is turned."""
    if stream is not None:
        with _on(stream, k):
            return cache_append(q, k, v, frequencies, k_pages, v_pages, block_table, start,
                                input_row_offsets=input_row_offsets, layout=layout, magnitude=magnitude, q_out=q_out)
    magnitude = float(magnitude)
    key = ("cache_append", _sig(q), _sig(k), _sig(v), _sig(frequencies), _sig(k_pages), _sig(v_pages),
           _sig(block_table), _sig(start), _sig(input_row_offsets), layout, magnitude, _sig(q_out))
    plan = _PLANS.get(key)
    if plan is None:
        pairs = _apart(_pairs((q_out, q, k, v, k_pages, v_pages), ("q_out", 0, 1, True), ("q_out", 0, 2), ("q_out", 0, 3),
                              ("q_out", 0, 4), ("q_out", 0, 5)), q_out, q, k, v, k_pages, v_pages)
        plan = _plan_append(key, q, k, v, frequencies, k_pages, v_pages, block_table, start, input_row_offsets,
                            layout, magnitude, q_out)
        plan.pairs, plan.pools = pairs, _pairs((k_pages, v_pages), ("k_pages", 0, 1))
        plan.reach = plan.pools[0][1] if plan.pools else 0
    elif plan.pairs:
        _apart(plan.pairs, q_out, q, k, v, k_pages, v_pages)
    keys, values = k_pages.data_ptr(), v_pages.data_ptr()
    if -plan.reach < keys - values < plan.reach:
        _apart(plan.pools, k_pages, v_pages)
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=plan.device)
    _call(plan, _p(q), k.data_ptr(), v.data_ptr(), _p(frequencies), keys, values, block_table.data_ptr(),
          start.data_ptr(), _p(input_row_offsets), _p(q_out))
    return q_out


def _plan_attention(key, q, k_pages, v_pages, block_table, lens, window, scale, softcap, span, slopes, out_dtype, out):
    dev = _device(q, k_pages, v_pages, block_table, lens, slopes, out)
    o_dtype = out.dtype if out is not None else (out_dtype or q.dtype)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out does not have out_dtype")
    if o_dtype not in _QKV_DTYPES:
        raise ValueError("the output dtype must be float32 or bfloat16")
    B = lens.numel()
    p = KdaCacheParams(window=window, span=span, scale=scale, softcap=softcap, o_dtype=_QKV_DTYPES[o_dtype])
    _pages(p, k_pages, v_pages, block_table, B)
    _index(lens, B, "lens")
    p.q_row_stride = _heads(q, "q")
    p.num_q_heads = q.shape[1]
    if q.shape[0] != B * window or q.shape[2] != p.head_dim or q.dtype != k_pages.dtype:
        raise ValueError("q must be [num_seqs * window, H, d] in the pages' dtype")
    if slopes is not None:
        _dense(slopes, (q.shape[1],), torch.float32, "slopes")
    if out is not None:
        _dense(out, q.shape, o_dtype, "out")
    n = ctypes.c_size_t(0)
    with torch.cuda.device(dev):
        st = _lib.load().kda_cache_attention_workspace_size(ctypes.byref(p), ctypes.byref(n))
    if st != _lib.KDA_OK:
        raise KdaError(st, "kda_cache_attention_workspace_size")
    return _keep(key, _Plan("kda_cache_attention", p, dev, n.value, q.shape, o_dtype))


def cache_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    block_table: torch.Tensor, lens: torch.Tensor, *, window: int = 1,
                    scale: float = 0.0, softcap: float = 0.0, span: int = 0,
                    slopes: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    return_lse: bool = False, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None):
    """Attention of the last `window` (1 to 64) tokens of each sequence over its cache
    (kda_cache_attention).  q [B * window, H, d], sequence by sequence, H a multiple of the pages'
    heads; lens [B] int32: the tokens in the cache, the window's own included (see `cache_append`).

    `scale` 0 means 1 / sqrt(d); `softcap` c: scores become c tanh(s / c); `slopes` [H] float32: adds
    slope * (key position - query position); `span` n: a query sees its own and the n - 1 keys before it (pages
    before those are not read).  Returns o [B * window, H, d] (q's dtype, or `out_dtype`), with
    `return_lse` (o, log of the sum of the exponentials [B * window, H] float32).  A query that sees
    nothing gets zeros and -inf.  `workspace` is not to be shared by calls that may run at the same time."""
    if stream is not None:
        with _on(stream, q):
            return cache_attention(q, k_pages, v_pages, block_table, lens, window=window, scale=scale,
                                   softcap=softcap, span=span, slopes=slopes, out_dtype=out_dtype,
                                   return_lse=return_lse, out=out, workspace=workspace)
    scale, softcap = float(scale), float(softcap)
    key = ("cache_attention", _sig16(q), _sig16(k_pages), _sig16(v_pages), _sig(block_table), _sig(lens), window, scale,
           softcap, span, _sig(slopes), out_dtype, _sig(out))
    plan = _PLANS.get(key)
    if plan is None:
        pairs = _apart(_pairs((out, q, k_pages, v_pages), ("out", 0, 1), ("out", 0, 2), ("out", 0, 3)), out, q, k_pages,
                       v_pages)
        plan = _plan_attention(key, q, k_pages, v_pages, block_table, lens, window, scale, softcap, span, slopes,
                               out_dtype, out)
        plan.pairs = pairs
    elif plan.pairs:
        _apart(plan.pairs, out, q, k_pages, v_pages)
    if out is None:
        out = torch.empty(plan.shape, dtype=plan.dtype, device=plan.device)
    lse = torch.empty(plan.shape[:2], dtype=torch.float32, device=plan.device) if return_lse else None
    space, address, nbytes = _space(plan, workspace)
    _call(plan, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
          _p(slopes), out.data_ptr(), _p(lse), address, nbytes)
    return (out, lse) if return_lse else out


# -------------------------------------------------------------------------------------------- tables

class CacheRows(NamedTuple):
    """What `cache_update` returns: the new tables, and the pages it copied."""
    table: torch.Tensor   # [S', max_pages] int32, -1 behind a row's pages
    lens: torch.Tensor    # [S']
    refs: torch.Tensor    # [num_pages]
    kept: torch.Tensor    # [S'] tokens that the row took over: where its new ones begin
    src: torch.Tensor     # [S'] pages to copy, then -1
    dst: torch.Tensor


class CacheMoves(NamedTuple):
    """What `cache_compact` returns."""
    table: torch.Tensor     # [S, max_pages] int32
    refs: torch.Tensor      # [num_pages]
    page_map: torch.Tensor  # [num_pages] where each page went, -1 for a free one
    src: torch.Tensor       # [num_pages / 2] pages that moved, then -1
    dst: torch.Tensor


def _plan_rows(key, name, block_table, lens, refs, parent, new_lens, page_size):
    dev = _device(block_table, lens, refs, parent, new_lens)
    S = lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != S or block_table.dtype != torch.int32 \
            or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [num_seqs, max_pages]")
    _index(lens, S, "lens")
    _index(refs, refs.numel(), "refs")
    out = S
    if new_lens is not None:
        out = new_lens.numel()
        _index(new_lens, out, "new_lens")
        if parent is not None:
            _index(parent, out, "parent")
        elif out != S:
            raise ValueError("without parent each row goes on from itself: new_lens must be shaped like lens")
    p = KdaCacheRowsParams(rows=S, rows_out=out, max_pages=block_table.shape[1], page_size=page_size,
                           num_pages=refs.numel())
    n = ctypes.c_size_t(0)
    st = _lib.load().kda_cache_rows_workspace_size(ctypes.byref(p), ctypes.byref(n))
    if st != _lib.KDA_OK:
        raise KdaError(st, "kda_cache_rows_workspace_size")
    return _keep(key, _Plan(name, p, dev, n.value, (out, block_table.shape[1])))


def _out(given, like, inputs):
    """The outputs that are given: of the shapes needed and of memory that no input and no other output has."""
    spans = [(t.data_ptr(), t.nbytes, None) for t in inputs if t is not None]
    for t, (name, shape) in zip(given, like):
        if t.shape != shape or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"out.{name} must be contiguous int32 {list(shape)}")
        spans.append((t.data_ptr(), t.nbytes, name))
    spans.sort(key=lambda x: x[0])
    end, out_end, last = 0, 0, None            # of all and of the outputs so far; the output that ends there
    for at, nbytes, name in spans:
        if nbytes and at < (out_end if name is None else end):
            raise ValueError(f"out.{name or last} must have memory of its own")
        if nbytes:
            end = max(end, at + nbytes)
            if name is not None:
                out_end, last = at + nbytes, name
    return given


def cache_update(block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                 parent: Optional[torch.Tensor], new_lens: torch.Tensor, *, page_size: int,
                 pools: Sequence[torch.Tensor] = (), out: Optional[CacheRows] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> CacheRows:
    """A cache's tables from one step to the next (kda_cache_update).  New row i goes on from row
    parent[i] (-1: from nothing; `parent` None: from row i) with its first
    min(lens[parent[i]], new_lens[i]) tokens and has pages for new_lens[i]: rows go on, fork, are cut
    back, grow, begin or end.  Full pages are shared; of the rows that end inside one page the lowest keeps it and
    the others get a copy.

    block_table [S, max_pages], lens [S], refs [num_pages] (references to each page; 0: free),
    parent and new_lens [S'], all int32.  `pools`: the layers' key and value pages, in which the copies
    are made (`cache_copy`); without them the caller makes them from `src` and `dst`.  The old tables stay valid.
    `out`: a `CacheRows` to write to, not the one that is read."""
    if stream is not None:
        with _on(stream, refs):
            return cache_update(block_table, lens, refs, parent, new_lens, page_size=page_size, pools=pools, out=out,
                                workspace=workspace)
    key = ("cache_update", _sig(block_table), _sig(lens), _sig(refs), _sig(parent), _sig(new_lens), page_size)
    plan = _PLANS.get(key)
    if plan is None:
        plan = _plan_rows(key, "kda_cache_update", block_table, lens, refs, parent, new_lens, page_size)
    (S, width), N, dev = plan.shape, plan.params.num_pages, plan.device
    if out is None:
        # one piece of memory for the tables: an allocation takes longer than the kernel's launch
        table, *rows = torch.empty(S * width + 4 * S + N, dtype=torch.int32, device=dev).split_with_sizes(
            [S * width, S, N, S, S, S])
        out = CacheRows(table.view(S, width), *rows)
    else:
        _device(refs, *out)
        _out(out, (("table", (S, width)), ("lens", (S,)), ("refs", (N,)), ("kept", (S,)), ("src", (S,)), ("dst", (S,))),
             (block_table, lens, refs, parent, new_lens))
    copy = _find_copy(pools, out.src, out.dst, N) if pools else None
    space, address, nbytes = _space(plan, workspace)
    _call(plan, block_table.data_ptr(), lens.data_ptr(), refs.data_ptr(), _p(parent), new_lens.data_ptr(),
          *[t.data_ptr() for t in out], address, nbytes)
    if copy is not None:
        _copy(copy, pools, out.src, out.dst)
    return out


def cache_compact(block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, *,
                  page_size: int, pools: Sequence[torch.Tensor] = (),
                  out: Optional[CacheMoves] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> CacheMoves:
    """Used pages to the front of the pools (kda_cache_compact): of n pages in use, the k-th from page n
    on goes to the k-th free page before n, in the tables and in `pools`.  Arguments as for
    `cache_update`; the old tables stay valid until a free page is written."""
    if stream is not None:
        with _on(stream, refs):
            return cache_compact(block_table, lens, refs, page_size=page_size, pools=pools, out=out,
                                 workspace=workspace)
    key = ("cache_compact", _sig(block_table), _sig(lens), _sig(refs), page_size)
    plan = _PLANS.get(key)
    if plan is None:
        plan = _plan_rows(key, "kda_cache_compact", block_table, lens, refs, None, None, page_size)
    shape, N, dev = plan.shape, plan.params.num_pages, plan.device
    if out is None:
        table, *rows = torch.empty(shape[0] * shape[1] + 2 * N + 2 * (N // 2), dtype=torch.int32, device=dev) \
            .split_with_sizes([shape[0] * shape[1], N, N, N // 2, N // 2])
        out = CacheMoves(table.view(shape), *rows)
    else:
        _device(refs, *out)
        _out(out, (("table", shape), ("refs", (N,)), ("page_map", (N,)), ("src", (N // 2,)), ("dst", (N // 2,))),
             (block_table, lens, refs))
    copy = _find_copy(pools, out.src, out.dst, N) if pools else None
    space, address, nbytes = _space(plan, workspace)
    _call(plan, block_table.data_ptr(), lens.data_ptr(), refs.data_ptr(), *[t.data_ptr() for t in out], address, nbytes)
    if copy is not None:
        _copy(copy, pools, out.src, out.dst)
    return out


class _Pools:
    """The host arrays of a `cache_copy` call but the pools' addresses, made once for each combination of shapes."""
    __slots__ = ("fn", "n", "entries", "sizes", "strides", "num_pages", "device", "index", "addresses")


def _plan_copy(key, pools, src, dst, num_pages):
    p = _Pools()
    p.device = _device(src, dst, *pools)
    _index(src, src.numel(), "src")
    _index(dst, src.numel(), "dst")
    p.num_pages = pools[0].shape[0] if num_pages is None else num_pages
    sizes, strides = [], []
    for t in pools:
        if t.dim() < 1 or t.shape[0] != p.num_pages or (t.shape[0] and not t[0].is_contiguous()) \
                or (t.shape[0] > 1 and t.stride(0) < t[0].numel()):
            raise ValueError(f"pools must be [{p.num_pages}, ...], each page one stretch of memory")
        size = t[0].numel() * t.element_size() if t.shape[0] else 0
        sizes.append(size)
        strides.append(t.stride(0) * t.element_size() if t.shape[0] > 1 else size)
    p.n, p.entries, p.index = len(pools), src.numel(), p.device.index
    p.sizes, p.strides = (ctypes.c_int64 * p.n)(*sizes), (ctypes.c_int64 * p.n)(*strides)
    p.addresses = ctypes.c_void_p * p.n
    p.fn = _lib.load().kda_cache_copy
    return _keep(key, p)


def _find_copy(pools, src, dst, num_pages=None):
    """The plan of a copy, its pools checked."""
    key = ("cache_copy", _sig(src), _sig(dst), num_pages, *[_sig(t) for t in pools])
    return _PLANS.get(key) or _plan_copy(key, pools, src, dst, num_pages)


def _copy(p, pools, src, dst):
    args = (p.addresses(*[t.data_ptr() for t in pools]), p.sizes, p.strides, p.n, src.data_ptr(), dst.data_ptr(),
            p.entries, p.num_pages)
    if _current_device() == p.index:
        st = p.fn(*args, _raw_stream(p.index))
    else:
        with torch.cuda.device(p.index):
            st = p.fn(*args, _raw_stream(p.index))
    if st != _lib.KDA_OK:
        raise KdaError(st, "kda_cache_copy")


def cache_copy(pools: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, *,
               stream: Optional[torch.cuda.Stream] = None) -> None:
    """pool[dst[i]] = pool[src[i]] in every pool (kda_cache_copy): pages of a cache, or slots of a recurrent state or
    convolution pool (a forked sequence's state); up to 64 neighbouring pools of one size go in one launch.
    src, dst [n] int32; the list ends at its first negative src, and every src behind it has to be
    negative.  No slot may be written twice or both read and written."""
    if not pools:
        return
    if stream is not None:
        with _on(stream, src):
            return cache_copy(pools, src, dst)
    _copy(_find_copy(pools, src, dst), pools, src, dst)
