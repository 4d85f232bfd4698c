"""Measured cases of the key-value cache of a hybrid model's attention layers.

  rotary, rotary_bwd  rotary positions of queries and keys, and the gradients' way back
  append              rotary positions of new tokens' queries and keys, the keys and values
                      written into the pages of a cache
  attention           one new token, or a window of draft tokens, per sequence over the pages
  update              a cache's page tables from one step to the next: rows continue, fork, are
                      cut back, grow or are freed; pages that may not be shared are copied
  compact             used pages moved to the front of the pools

`run` computes them in elementary torch operations in fp32 (own = False) or through the library's
entry points (own = True); `exact` evaluates the definitions in fp64, each written on its own.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}


# ------------------------------------------------------------------------------------------ cases

def _rotary(name, op, T, H, HK, D, R, dtype=BF16, layout="half", scaling="none", packed=False):
    return dict(name=name, op=op, T=T, H=H, HK=HK, D=D, R=R, dtype=dtype, layout=layout,
                scaling=scaling, packed=packed)


def _append(name, B, lo, hi, past_lo, past_hi, H, HK, D, R, P, dtype=BF16, layout="half",
            scaling="none"):
    """B sequences that hold past_lo .. past_hi tokens and get lo .. hi new ones."""
    return dict(name=name, op="append", B=B, lo=lo, hi=hi, past_lo=past_lo, past_hi=past_hi, H=H,
                HK=HK, D=D, R=R, P=P, dtype=dtype, layout=layout, scaling=scaling)


def _attention(name, B, lo, hi, H, HK, D, P, W=1, dtype=BF16, out=None, softcap=0.0, span=0,
               slopes=False, lse=False, empty=0):
    """B sequences of lo .. hi tokens, the last W of each being its queries; the first `empty` of
    them hold nothing."""
    return dict(name=name, op="attention", B=B, lo=lo, hi=hi, H=H, HK=HK, D=D, P=P, W=W,
                dtype=dtype, out=out or dtype, softcap=softcap, span=span, slopes=slopes, lse=lse,
                empty=empty)


def _update(name, kind, S, lo, hi, P, HK, D, pools, branch=1, grow=1, dtype=BF16):
    """kind "step": S rows go on by `grow` tokens, one in 16 ends and one in 16 is new; "fork":
    S rows become S * branch, each parent's continuations growing by `grow`; "beam": S rows each
    continue a row of their group of `branch`."""
    return dict(name=name, op="update", kind=kind, S=S, lo=lo, hi=hi, P=P, HK=HK, D=D,
                pools=pools, branch=branch, grow=grow, dtype=dtype)


def _compact(name, S, lo, hi, P, HK, D, pools, spread=2.0, dtype=BF16):
    """S rows whose pages lie scattered over `spread` times as many."""
    return dict(name=name, op="compact", S=S, lo=lo, hi=hi, P=P, HK=HK, D=D, pools=pools,
                spread=spread, dtype=dtype)


def listed():
    return [
        # the rotation in one training step of 4 x 4096 tokens, 32 query and 8 key heads
        _rotary("rotary_train", "rotary", 16384, 32, 8, 128, 128),
        # its gradients for a small fp32 model: part of an odd head rotated, adjacent pairs, the
        # frequencies of a lengthened context
        _rotary("rotary_bwd_part_f32", "rotary_bwd", 4099, 7, 7, 100, 50, dtype=F32,
                layout="interleaved", scaling="by_parts"),
        # a decode step of 256 sequences: one token each into its page
        _append("append_decode", 256, 1, 1, 1, 1000, 32, 8, 128, 128, 16),
        # a ragged prompt batch behind far positions, half of each head rotated
        _append("append_prompts", 8, 200, 8192, 1, 1000000, 16, 16, 128, 64, 64, layout="interleaved",
                scaling="ntk"),
        # one user's next token, the latency of a single call
        _attention("attention_one_user", 1, 5000, 5000, 16, 2, 128, 16, lse=True),
        # a decode batch of 256 ragged sequences: the cache is the work
        _attention("attention_decode_256", 256, 256, 8192, 32, 8, 128, 64),
        # few sequences with very long caches, split over the whole GPU
        _attention("attention_long", 3, 120001, 262144, 16, 4, 128, 16, softcap=50.0, out=F32),
        # the window of a speculative decoder over a small fp32 model with odd pages, distance
        # bias, a sequence that has just been freed
        _attention("attention_drafts_f32", 61, 3, 3000, 8, 4, 80, 24, W=4, dtype=F32, slopes=True,
                   span=1024, lse=True, empty=2),
        # the tables of a serving batch from one decode step to the next
        _update("update_step", "step", 256, 1, 4000, 16, 2, 64, 2),
        # eight continuations of each prompt: whole pages shared, the open page of each copied
        _update("update_fork", "fork", 64, 2000, 16000, 16, 4, 128, 8, branch=8, grow=4),
        # a small pool after its sequences have come and gone
        _compact("compact_small", 16, 1, 700, 16, 2, 64, 2),
        # the pools of four layers, half empty
        _compact("compact_layers", 128, 500, 6000, 32, 4, 128, 8),
    ]


_MAX_BYTES, _MAX_FLOPS = 2 << 30, 8 << 30


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_bwd", "append", "append", "attention", "attention",
                     "attention", "attention", "update", "compact"])
    dtype = rng.choice([BF16, BF16, F32])
    D = rng.choice([128, 128, 64, 256, 80, 16])
    HK = rng.choice([1, 2, 4, 8])
    H = HK * rng.choice([1, 2, 4, 7, 8])
    P = rng.choice([16, 16, 64, 32, 24, 128, 1])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
    if op in ("rotary", "rotary_bwd"):
        D = rng.choice([128, 64, 256, 100, 38, 16])
        R = rng.choice([D, D, D // 4 * 2])
        T = _log_int(rng, 1, 16384)
        while T * (H + HK) * D * _SIZE[dtype] > 320 << 20:
            T = T * 3 // 4
        return _unnamed(_rotary(None, op, T, H, HK, D, R, dtype, layout, scaling,
                                rng.random() < 0.5))
    if op == "append":
        R = rng.choice([D, D, D // 4 * 2])
        B = _log_int(rng, 1, 512)
        hi = rng.choice([1, 4, _log_int(rng, 2, 8192)])
        while B * hi * (H + 2 * HK) * D * _SIZE[dtype] > 320 << 20:
            B, hi = max(1, B // 2), max(1, hi * 3 // 4)
        past = _log_int(rng, 2, min(1000000, (1 << 24) * P // B))
        return _unnamed(_append(None, B, (hi + 1) // 2, hi, 1, past, H, HK, D, R, P, dtype, layout,
                                scaling))
    if op == "attention":
        W = rng.choice([1, 1, 1, 2, 5, 8])
        B = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, 262144)
        while B * hi * HK * D * _SIZE[dtype] * 2 > _MAX_BYTES or 4 * B * hi * H * W * D > _MAX_FLOPS:
            B, hi = max(1, B * 2 // 3), max(1, hi * 3 // 4)
        return _unnamed(_attention(None, B, max(1, hi // rng.choice([1, 3, 20])), hi, H, HK, D, P, W,
                                   dtype, rng.choice([dtype, F32]), rng.choice([0.0, 0.0, 30.0]),
                                   rng.choice([0, 0, _log_int(rng, 1, hi + 1)]),
                                   rng.random() < 0.3, rng.random() < 0.5,
                                   rng.choice([0, 0, 1]) if B > 1 else 0))
    S = _log_int(rng, 1, 512)
    hi = _log_int(rng, 1, 16000)
    pools = rng.choice([2, 4, 8, 16])
    while S * (3 * hi + 10 * (P + 100)) * HK * D * _SIZE[dtype] * pools > _MAX_BYTES:
        S, hi, pools = max(1, S * 2 // 3), max(1, hi * 2 // 3), max(2, pools // 2)
    lo = max(1, hi // 8)
    if op == "update":
        kind = rng.choice(["step", "fork", "beam"])
        branch = 1 if kind == "step" else rng.choice([2, 4, 5])
        S = max(1, S // branch) * (branch if kind == "beam" else 1)
        return _unnamed(_update(None, kind, S, lo, hi, P, HK, D, pools, branch,
                                rng.choice([1, 1, 5, 100]), dtype))
    return _unnamed(_compact(None, S, lo, hi, P, HK, D, pools, rng.choice([1.25, 2.0, 3.0]), dtype))


def _unnamed(case):
    del case["name"]
    return case


# A case's lengths and parents are the same for every seed (they set the work); where its pages lie
# and what they hold differ from seed to seed.

def _rng_of(case, what):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + what)


def _lengths(case, n, lo, hi, what):
    r = _rng_of(case, what)
    return [min(hi, max(lo, _log_int(r, lo, hi))) for _ in range(n)]


def _attention_lens(case):
    e = case["empty"]
    return [0] * e + _lengths(case, case["B"] - e, case["lo"], case["hi"], "lens")


def _first_visible(case, length):
    """The first key that any query of the sequence sees."""
    return max(0, length - case["W"] - case["span"] + 1) if case["span"] else 0


def _rows_of(case):
    """The rows before and after an update: lengths, parents and new lengths."""
    S, br = case["S"], case["branch"]
    lens = _lengths(case, S, case["lo"], case["hi"], "lens")
    r = _rng_of(case, "parents")
    parent, new = [], []
    if case["kind"] == "step":
        for i in range(S):
            ends, fresh = r.random() < 1 / 16, r.random() < 1 / 16
            parent.append(-1 if ends or fresh else i)
            new.append(0 if ends else _log_int(r, case["lo"], case["hi"]) if fresh else lens[i] + case["grow"])
    elif case["kind"] == "fork":
        for i in range(S * br):
            parent.append(i // br)
            new.append(lens[i // br] + case["grow"])
    else:
        for i in range(S):                      # a group's beams have one length
            lens[i] = lens[i // br * br]
        for i in range(S):
            parent.append(i // br * br + r.randrange(br))
            new.append(lens[i] + case["grow"])
    return lens, parent, new


# ----------------------------------------------------------------------------------------- inputs

def _frequencies(R, scaling, base=10000.0):
    """Radians per position of each pair, and the factor of the rotated values: plain; positions
    interpolated; base raised; or interpolated where a pair turns less than once over the
    context it was trained on, kept where it turns more than 32 times, blended between."""
    factor, trained = 8.0, 4096
    if scaling == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "by_parts":
        share = [min(1.0, max(0.0, (trained * x / (2 * math.pi) - 1) / 31)) for x in f]
        return [x * a + x / factor * (1 - a) for x, a in zip(f, share)], 0.1 * math.log(factor) + 1
    return f, 1.0


def _long(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(lens, P):
    return [-(-n // P) for n in lens]


def _place(gen, spans, width, num_pages, skip=None):
    """A page table [rows, width]: each row's pages at random places of the pool, -1 behind them
    and in the first skip[row] entries."""
    skip = skip or [0] * len(spans)
    order = torch.randperm(num_pages, generator=gen, device=DEV).to(torch.int32)
    n, k = torch.tensor(spans, device=DEV), torch.tensor(skip, device=DEV)
    col = torch.arange(width, device=DEV)
    first = torch.cumsum(n - k, 0) - (n - k)
    at = first[:, None] + col[None] - k[:, None]
    live = (col[None] >= k[:, None]) & (col[None] < n[:, None])
    table = torch.where(live, order[at.clamp(0, num_pages - 1)], -1)
    return table.to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dt)

    s = dict(case)
    op, D, HK = case["op"], case["D"], case["HK"]
    if "R" in case:
        f, s["magnitude"] = _frequencies(case["R"], case["scaling"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if op in ("rotary", "rotary_bwd"):
        T, H = case["T"], case["H"]
        if case["packed"]:                      # column blocks of a packed [Q | K | V] projection
            x = normal(T, (H + 2 * HK) * D)
            s["q"] = x[:, :H * D].unflatten(1, (H, D))
            s["k"] = x[:, H * D:(H + HK) * D].unflatten(1, (HK, D))
        else:
            s["q"], s["k"] = normal(T, H, D), normal(T, HK, D)
        # ragged prompts, some of them continuing far behind the start
        cut = torch.rand(T, generator=gen, device=DEV) < 1 / 700
        start = torch.randint(0, 1000000, (T,), generator=gen, device=DEV)
        at = torch.arange(T, device=DEV)
        head = torch.cummax(torch.where(cut, at, 0), 0).values
        s["positions"] = at - head + torch.where(cut[head], start[head], 0)
    elif op == "append":
        B, P, H = case["B"], case["P"], case["H"]
        new = _lengths(case, B, case["lo"], case["hi"], "new")
        past = _lengths(case, B, case["past_lo"], case["past_hi"], "past")
        n = _pages([a + b for a, b in zip(past, new)], P)
        # pages more than 1000 tokens behind are no longer held
        skip = [max(0, a - 1000) // P for a in past]
        num = sum(n) - sum(skip) + 7
        s["table"] = _place(gen, n, max(n), num, skip)
        s["k_pages"], s["v_pages"] = normal(num, P, HK, D), normal(num, P, HK, D)
        T = sum(new)
        s["q"], s["k"], s["v"] = normal(T, H, D), normal(T, HK, D), normal(T, HK, D)
        s["start"] = _long(past)
        s["offsets"] = _long([0] + list(np.cumsum(new)))
    elif op == "attention":
        B, P = case["B"], case["P"]
        lens = _attention_lens(case)
        n = _pages(lens, P)
        skip = [_first_visible(case, x) // P for x in lens]
        num = sum(n) - sum(skip) + 3
        s["table"] = _place(gen, n, max(1, max(n)), num, skip)
        s["k_pages"], s["v_pages"] = normal(num, P, HK, D), normal(num, P, HK, D)
        s["q"] = normal(B * case["W"], case["H"], D)
        s["lens"] = _long(lens)
        s["slopes_t"] = None
        if case["slopes"]:
            s["slopes_t"] = torch.rand(case["H"], generator=gen, device=DEV) * 0.02
    else:
        P, S = case["P"], case["S"]
        if op == "update":
            lens, parent, new = _rows_of(case)
            s["parent"], s["new_lens"] = _long(parent), _long(new)
            kept = [min(lens[p], w) if p >= 0 else 0 for p, w in zip(parent, new)]
            room = sum(_pages(lens, P)) + sum(_pages(new, P)) - sum(k // P for k in kept) + 5
            width = max(1, max(_pages(lens + new, P)))
        else:
            lens = _lengths(case, S, case["lo"], case["hi"], "lens")
            room = int(sum(_pages(lens, P)) * case["spread"]) + 5
            width = max(_pages(lens, P))
        s["lens"] = _long(lens)
        s["table"] = _place(gen, _pages(lens, P), width, room)
        s["refs"] = torch.zeros(room + 1, dtype=torch.int32, device=DEV).index_add_(
            0, torch.where(s["table"] < 0, room, s["table"]).flatten().long(),
            torch.ones(s["table"].numel(), dtype=torch.int32, device=DEV))[:room].contiguous()
        s["stack"] = normal(case["pools"], room, P, HK, D)
        s["pool_list"] = list(s["stack"].unbind(0))
    return s


# -------------------------------------------------------------------------------------- plain form

def _turn(x, positions, s, sign):
    """x [T, heads, D] rotated by sign times its positions' angles (angles in fp64: far positions),
    in fp32."""
    R = s["R"]
    angle = positions.double()[:, None, None] * s["freq"]
    c = (s["magnitude"] * torch.cos(angle)).float()
    d = (s["magnitude"] * sign * torch.sin(angle)).float()
    x = x.float()
    if s["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * d, b * c + a * d], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rotary(s):
    sign = 1 if s["op"] == "rotary" else -1
    return [_turn(s[n], s["positions"], s, sign).to(s[n].dtype) for n in ("q", "k")]


def _plain_append(s):
    P = s["P"]
    T = s["q"].shape[0]
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["offsets"][1:].long(), t, right=True)
    pos = s["start"].long()[seq] + t - s["offsets"].long()[seq]
    page = s["table"].long()[seq, pos // P]
    s["k_pages"][page, pos % P] = _turn(s["k"], pos, s, 1).to(s["k"].dtype)
    s["v_pages"][page, pos % P] = s["v"]
    return _turn(s["q"], pos, s, 1).to(s["q"].dtype), s["k_pages"], s["v_pages"]


def _plain_attention(s):
    B, W, H, HK, D, P = (s[n] for n in ("B", "W", "H", "HK", "D", "P"))
    width = s["table"].shape[1]
    at = s["table"].long().clamp(min=0)
    k = s["k_pages"][at].view(B, width * P, HK, D).permute(0, 2, 3, 1).float()
    v = s["v_pages"][at].view(B, width * P, HK, D).transpose(1, 2).float()
    q = s["q"].view(B, W, HK, H // HK, D).permute(0, 2, 1, 3, 4).float()
    x = (q.reshape(B, HK, -1, D) @ k).view(B, HK, W, H // HK, -1) / math.sqrt(D)
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    pos = (s["lens"].long()[:, None] - W + torch.arange(W, device=DEV))[:, None, :, None, None]
    j = torch.arange(width * P, device=DEV)
    if s["slopes_t"] is not None:
        x = x + s["slopes_t"].view(HK, 1, H // HK, 1) * (j - pos)
    seen = j <= pos
    if s["span"]:
        seen = seen & (j > pos - s["span"])
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    # rows behind a sequence's end may lie in pages of others: their weight is zero
    o = (e.reshape(B, HK, -1, width * P) @ v).view(B, HK, W, H // HK, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * W, H, D).to(_DT[s["out"]])
    if not s["lse"]:
        return o
    return o, (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B * W, H)


def _plain_update(s):
    P, N = s["P"], s["refs"].numel()
    table, lens, parent, new = (s[n].long() for n in ("table", "lens", "parent", "new_lens"))
    width = table.shape[1]
    col = torch.arange(width, device=DEV)
    # references that stay: those from elsewhere and those of whole pages
    others = torch.zeros(N + 1, dtype=torch.long, device=DEV)
    others[:N] = s["refs"]
    held = torch.where(col < ((lens + P - 1) // P)[:, None], table, N)
    others.scatter_add_(0, held.flatten(), torch.full((held.numel(),), -1, device=DEV))
    old = parent.clamp(min=0)
    kept = torch.where(parent >= 0, torch.minimum(lens[old], new), 0)
    rows, whole = table[old], kept // P
    shared = torch.where(col < whole[:, None], rows, N)
    others.scatter_add_(0, shared.flatten(), torch.ones(shared.numel(), dtype=torch.long, device=DEV))
    # a page that ends inside its last token: the first row that holds it keeps it if no other may read it
    opened = kept % P != 0
    page = torch.where(opened, rows.gather(1, whole.clamp(max=width - 1)[:, None])[:, 0], N)
    row = torch.arange(parent.numel(), device=DEV)
    first = torch.full((N + 1,), parent.numel(), device=DEV).scatter_reduce_(0, page, row, "amin")
    stays = opened & (others[page] == 0) & (first[page] == row)
    have, want = whole + stays, (new + P - 1) // P
    need = want - have
    free = torch.argsort((s["refs"] != 0).to(torch.int8), stable=True)
    fresh = free[((torch.cumsum(need, 0) - need)[:, None] + col - have[:, None]).clamp(0, N - 1)]
    is_new = (col >= have[:, None]) & (col < want[:, None])
    out = torch.where(col < have[:, None], rows, torch.where(is_new, fresh, -1))
    for_refs = torch.where(is_new, fresh, N).flatten()
    others.scatter_add_(0, for_refs, torch.ones_like(for_refs))
    others.scatter_add_(0, torch.where(stays, page, N), torch.ones_like(page))
    copied = (opened & ~stays).nonzero()[:, 0]
    s["stack"][:, out[copied, whole[copied]]] = s["stack"][:, page[copied]]
    i32 = torch.int32
    return {"table": out.to(i32), "lens": new.to(i32), "refs": others[:N].to(i32),
            "kept": kept.to(i32), "pools": s["stack"]}


def _plain_compact(s):
    P, N = s["P"], s["refs"].numel()
    used = s["refs"] > 0
    at = torch.arange(N, device=DEV)
    front = at < used.sum()
    source, target = (used & ~front).nonzero()[:, 0], (~used & front).nonzero()[:, 0]
    where = torch.where(used, at, -1)
    where[source] = target
    refs = torch.where(front, s["refs"], 0)
    refs[target] = s["refs"][source]
    s["stack"][:, target] = s["stack"][:, source]
    live = torch.arange(s["table"].shape[1], device=DEV) < ((s["lens"] + P - 1) // P)[:, None]
    table = torch.where(live, where[s["table"].long().clamp(min=0)], -1)
    return {"table": table.to(torch.int32), "refs": refs, "page_map": where.to(torch.int32),
            "pools": s["stack"]}


# ------------------------------------------------------------------------------------ library calls

def _own_run(s):
    import gated_delta_rule_deltanet_gb300 as kda
    op = s["op"]
    if op in ("rotary", "rotary_bwd"):
        call = kda.rotary if op == "rotary" else kda.rotary_bwd
        return list(call(s["q"], s["k"], s["positions"], s["freq"], layout=s["layout"],
                         magnitude=s["magnitude"]))
    if op == "append":
        q = kda.cache_append(s["q"], s["k"], s["v"], s["freq"], s["k_pages"], s["v_pages"],
                             s["table"], s["start"], input_row_offsets=s["offsets"],
                             layout=s["layout"], magnitude=s["magnitude"])
        return q, s["k_pages"], s["v_pages"]
    if op == "attention":
        return kda.cache_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                   window=s["W"], softcap=s["softcap"], span=s["span"],
                                   slopes=s["slopes_t"], out_dtype=_DT[s["out"]],
                                   return_lse=s["lse"])
    if op == "update":
        r = kda.cache_update(s["table"], s["lens"], s["refs"], s["parent"], s["new_lens"],
                             page_size=s["P"], pools=s["pool_list"])
        return {"table": r.table, "lens": r.lens, "refs": r.refs, "kept": r.kept,
                "pools": s["stack"]}
    r = kda.cache_compact(s["table"], s["lens"], s["refs"], page_size=s["P"], pools=s["pool_list"])
    return {"table": r.table, "refs": r.refs, "page_map": r.page_map, "pools": s["stack"]}


def run(state):
    if own:
        return _own_run(state)
    return {"rotary": _plain_rotary, "rotary_bwd": _plain_rotary, "append": _plain_append,
            "attention": _plain_attention, "update": _plain_update,
            "compact": _plain_compact}[state["op"]](state)


# -------------------------------------------------------------------------------------------- work

def work(case):
    op, D, HK, e = case["op"], case["D"], case["HK"], _SIZE[case["dtype"]]
    if op in ("rotary", "rotary_bwd"):
        T, heads = case["T"], case["H"] + HK
        return {"bytes": 2 * T * heads * D * e + 8 * T + 4 * case["R"], "flops": 3 * T * heads * case["R"]}
    if op == "append":
        T = sum(_lengths(case, case["B"], case["lo"], case["hi"], "new"))
        return {"bytes": 2 * T * (case["H"] + 2 * HK) * D * e + 8 * T + 8 * case["B"] + 4 * case["R"],
                "flops": 3 * T * (case["H"] + HK) * case["R"]}
    if op == "attention":
        W, H, B = case["W"], case["H"], case["B"]
        keys = sum(n - _first_visible(case, n) for n in _attention_lens(case))
        b = keys * HK * D * 2 * e + 4 * (keys // case["P"] + B)
        b += B * W * H * (D * (e + _SIZE[case["out"]]) + 4 * case["lse"])
        return {"bytes": b, "flops": 4 * D * H * W * keys}
    P, page = case["P"], case["P"] * HK * D * e * case["pools"]
    if op == "update":
        lens, parent, new = _rows_of(case)
        n, m, entries = sum(_pages(lens, P)), sum(_pages(new, P)), len(new) * max(_pages(lens + new, P))
        copies = sum(p >= 0 and min(lens[p], w) % P != 0 and p in parent[:i]
                     for i, (p, w) in enumerate(zip(parent, new)))
        return {"bytes": 4 * (n + entries) + 8 * (n + m + 5) + 2 * copies * page, "flops": n + entries}
    lens = _lengths(case, case["S"], case["lo"], case["hi"], "lens")
    n, pages = sum(_pages(lens, P)), int(sum(_pages(lens, P)) * case["spread"]) + 5
    # the used pages lie at random: of the n at the front, the share of free ones moves in
    moved = int(n * (pages - n) / pages)
    b = 4 * (n + case["S"] * max(_pages(lens, P))) + 12 * pages + 2 * moved * page
    return {"bytes": b, "flops": n + pages}


# ------------------------------------------------------------------------------------------- exact

def _exact_turn(x, positions, case, sign):
    f, magnitude = _frequencies(case["R"], case["scaling"])
    R, y = case["R"], x.double().clone()
    turn = torch.polar(torch.tensor(magnitude, dtype=torch.float64, device=DEV),
                       sign * torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64, device=DEV)))
    first = torch.arange(R // 2, device=DEV) * (1 if case["layout"] == "half" else 2)
    second = first + (R // 2 if case["layout"] == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None, :]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(case, s):
    """An update's or a compaction's tables, row by row on the host."""
    P = case["P"]
    table, lens, refs = (s[n].tolist() for n in ("table", "lens", "refs"))
    if len(table) * len(table[0]) * case.get("branch", 1) > 1 << 22:
        return None                             # minutes of host time
    copies = []
    if case["op"] == "compact":
        used = [q for q, r in enumerate(refs) if r]
        kept_pages = set(q for q in used if q < len(used))
        holes = [q for q in range(len(used)) if q not in kept_pages]
        goes = {q: q for q in kept_pages}
        for q, h in zip([q for q in used if q >= len(used)], holes):
            goes[q] = h
            copies.append((q, h))
        new_refs = [0] * len(refs)
        for q, h in goes.items():
            new_refs[h] = refs[q]
        rows = [[goes[q] for q in r[:-(-n // P)]] for r, n in zip(table, lens)]
        out = {"refs": new_refs, "page_map": [goes.get(q, -1) for q in range(len(refs))]}
    else:
        parent, new = s["parent"].tolist(), s["new_lens"].tolist()
        free = iter([q for q, r in enumerate(refs) if r == 0])
        count = list(refs)
        for r, n in zip(table, lens):
            for q in r[:-(-n // P)]:
                count[q] -= 1
        kept = [min(lens[p], w) if p >= 0 else 0 for p, w in zip(parent, new)]
        rows = [list(table[p][:k // P]) if p >= 0 else [] for p, k in zip(parent, kept)]
        for r in rows:
            for q in r:
                count[q] += 1
        claimed = set()
        for i, (p, k, w) in enumerate(zip(parent, kept, new)):
            if k % P:
                q = table[p][k // P]
                if count[q] == 0 and q not in claimed:
                    claimed.add(q)
                    rows[i].append(q)
                else:
                    h = next(free)
                    copies.append((q, h))
                    rows[i].append(h)
                    count[h] = 1
            while len(rows[i]) < -(-w // P):
                h = next(free)
                rows[i].append(h)
                count[h] = 1
        for q in claimed:
            count[q] += 1
        out = {"lens": new, "refs": count, "kept": kept}
    out["table"] = [r + [-1] * (s["table"].shape[1] - len(r)) for r in rows]
    out = {k: torch.tensor(v, dtype=torch.int32) for k, v in out.items()}
    if copies:
        a, b = torch.tensor(copies, device=DEV).unbind(1)
        s["stack"].index_copy_(1, b, s["stack"].index_select(1, a))
    out["pools"] = s["stack"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "rotary_bwd"):
        sign = 1 if op == "rotary" else -1
        return [_exact_turn(s[n], s["positions"], case, sign) for n in ("q", "k")]
    if op == "append":
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        offsets, start, table = (s[n].tolist() for n in ("offsets", "start", "table"))
        pos = torch.cat([torch.arange(b - a) + p for a, b, p in zip(offsets, offsets[1:], start)])
        page = [table[i][p // case["P"]] for i, (a, b, f) in enumerate(zip(offsets, offsets[1:], start))
                for p in range(f, f + b - a)]
        page, pos = torch.tensor(page, device=DEV), pos.to(DEV)
        k_pages[page, pos % case["P"]] = _exact_turn(s["k"], pos, case, 1)
        v_pages[page, pos % case["P"]] = s["v"].double()
        return _exact_turn(s["q"], pos, case, 1), k_pages, v_pages
    if op in ("update", "compact"):
        return _exact_rows(case, s)
    W, H, HK, D, P = (case[n] for n in ("W", "H", "HK", "D", "P"))
    o = torch.zeros(case["B"] * W, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"] * W, H), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_attention_lens(case)):
        lo = _first_visible(case, n)
        if n == 0:
            continue
        j = torch.arange(lo, n, device=DEV)
        page = s["table"][b].long()[j // P]
        k, v = s["k_pages"][page, j % P].double(), s["v_pages"][page, j % P].double()
        for w in range(W):
            p = n - W + w
            a = max(0, p - case["span"] + 1) if case["span"] else 0
            if p < a:
                continue
            seen = slice(a - lo, p + 1 - lo)
            q = s["q"][b * W + w].double().view(HK, H // HK, D)
            x = torch.einsum("hgd,jhd->hgj", q, k[seen]) * D ** -0.5
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if case["slopes"]:
                x = x + s["slopes_t"].double().view(HK, -1, 1) * (j[seen] - p)
            lse[b * W + w] = torch.logsumexp(x, -1).flatten()
            o[b * W + w] = torch.einsum("hgj,jhd->hgd", torch.softmax(x, -1), v[seen]).reshape(H, D)
    return (o, lse) if case["lse"] else o
