"""The layer's operators together, as a model runs them: norm, projections, front end,
recurrence, output norm and projection; and how they are launched: streams, graphs, workspaces.

A run is checked stage by stage: every operator's output against the fp64 reference of that
operator on the values the GPU handed to it, so that no tolerance has to cover more than one
operator (those of `test_gpu_layer.py`, `test_gpu_conv.py` and `test_gpu_parity.py`).
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_deltanet_gb300 as kda
import oracle
import workloads
from gated_delta_rule_deltanet_gb300 import _lib, layer
from oracle import conv as oc
from oracle import layer as ol
from test_gpu_layer import DEV, U, check, dev, host, no_error, product_tol, rng
from workloads import torch_io

pytestmark = pytest.mark.gpu


def rel(x, ref):
    return float(np.max(np.abs(x - ref)) / np.max(np.abs(ref)))


class Model:
    """One layer: residual stream [T, N] fp32, N = HV * d, bf16 activations."""

    def __init__(self, seed, HK=2, HV=4, d=128, W=4, per_channel=True):
        r = rng(seed)
        self.HK, self.HV, self.d, self.per_channel = HK, HV, d, per_channel
        N, CD = HV * d, (2 * HK + HV) * d
        ga = HV * d if per_channel else HV

        def w(rows, cols):
            return dev(r.standard_normal((rows, cols)) / np.sqrt(cols), "bf16")[0]

        def v(n, mean, std):
            return dev(mean + std * r.standard_normal(n), "f32")[0]
        self.post_w, self.pre_w, self.res_gate = v(N, 1, .1), v(N, 1, .1), v(N, .5, .1)
        self.w_in, self.w_a, self.w_b, self.w_g, self.w_o = w(CD, N), w(ga, N), w(HV, N), w(N, N), w(N, N)
        self.a_bias, self.b_bias = v(ga, 0, .1), v(HV, 0, .1)
        self.conv_w, self.conv_b = v((CD, W), 0, .5), v(CD, 0, .1)
        self.A_log = torch.full((HV,), float(np.log(0.05)), device=DEV)
        self.out_w = v(d, 1, .1)

    def run(self, block, stream, conv_state, pool, slots, offsets=None):
        """`block`: the previous block's output [T, N] bf16; `stream`: the residual stream before
        it.  Returns every stage's output."""
        m, T = self, block.shape[0]
        s = {}
        s["y"], s["h"] = kda.residual_norm(block, m.pre_w, residual=stream, post_weight=m.post_w,
                                           gate=m.res_gate, scale=0.5)
        s["proj"] = kda.linear(s["y"], m.w_in)
        s["a"] = kda.linear(s["y"], m.w_a, m.a_bias, out_dtype=torch.float32)
        s["b"] = kda.linear(s["y"], m.w_b, m.b_bias, out_dtype=torch.float32)
        s["gate"] = kda.linear(s["y"], m.w_g)
        a = s["a"].view(T, m.HV, m.d) if m.per_channel else s["a"]
        qkv, s["g"], s["beta"] = kda.conv_gates(
            s["proj"], m.conv_w, a, s["b"], num_k_heads=m.HK, num_v_heads=m.HV, d=m.d,
            conv_bias=m.conv_b, A_log=m.A_log, input_row_offsets=offsets, slot_idx=slots,
            conv_state=conv_state)
        s["qkv"] = qkv
        kd = m.HK * m.d
        q, k = qkv[:, :kd].view(T, m.HK, m.d), qkv[:, kd:2 * kd].view(T, m.HK, m.d)
        v = qkv[:, 2 * kd:].view(T, m.HV, m.d)
        if offsets is None:
            s["o"] = kda.decode_step(q, k, v, s["beta"], s["g"], slots, pool)
        else:
            s["o"] = kda.prefill(q, k, v, s["beta"], s["g"], offsets, slots, pool)
        s["z"] = kda.gated_norm(s["o"], s["gate"].view(T, m.HV, m.d), m.out_w, activation="silu")
        s["out"] = kda.linear(s["z"].view(T, -1), m.w_o, residual=s["h"], out_dtype=torch.float32)
        return s


def i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


@pytest.mark.parametrize("per_channel", [False, True])
def test_layer_stage_by_stage(per_channel):
    lens = [70, 0, 1, 130]
    m = Model(1, per_channel=per_channel)
    r = rng(2)
    T, N, CD = sum(lens), m.HV * m.d, m.w_in.shape[0]
    block, block64 = dev(r.standard_normal((T, N)), "bf16")
    stream, stream64 = dev(r.standard_normal((T, N)), "f32")
    conv_state, conv64 = dev(r.standard_normal((6, CD, 3)), "bf16")
    pool, pool64 = dev(r.standard_normal((6, m.HV, m.d, m.d)) * 0.02, "f32")
    off, slots = np.concatenate([[0], np.cumsum(lens)]), np.array([4, 0, 2, 5])
    s = m.run(block, stream, conv_state, pool, i32(slots), i32(off))
    no_error()
    y_ref, h_ref = ol.residual_norm(block64, host(m.pre_w), stream64, host(m.post_w), host(m.res_gate), 0.5)
    terms = np.abs(stream64) + np.abs(h_ref - stream64)
    check("h", s["h"], h_ref, 64 * U * terms)
    check("y", s["y"], y_ref, 128 * U * terms * ol.rms(h_ref, 1e-6)[1] * host(m.pre_w) + 64 * U * np.abs(y_ref))
    y = host(s["y"])
    for name, w, b in (("proj", m.w_in, None), ("a", m.w_a, m.a_bias), ("b", m.w_b, m.b_bias),
                       ("gate", m.w_g, None)):
        ref = ol.linear(y, host(w), None if b is None else host(b))[0]
        check(name, s[name], ref, product_tol(y, host(w).T, N, "bf16") + 4 * U * np.abs(ref))
    a = host(s["a"])
    qkv_ref, g_ref, beta_ref, _ = oc.conv_gates(
        x=host(s["proj"]), weight=host(m.conv_w), bias=host(m.conv_b),
        a=a.reshape(T, m.HV, m.d) if per_channel else a, b=host(s["b"]), A_log=host(m.A_log), dt_bias=None,
        offsets=off, slot_idx=slots, conv_state=conv64, num_v_heads=m.HV, per_channel=per_channel)
    assert rel(host(s["qkv"]), qkv_ref) <= 2e-3 + 2.0 ** -8
    assert rel(host(s["g"]), g_ref) <= 1e-5 and rel(host(s["beta"]), beta_ref) <= 1e-5
    qkv, kd = host(s["qkv"]), m.HK * m.d
    o_ref, _ = oracle.run_arrays(
        offsets=off, slot_idx=slots, q=qkv[:, :kd].reshape(T, m.HK, m.d),
        k=qkv[:, kd:2 * kd].reshape(T, m.HK, m.d), v=qkv[:, 2 * kd:].reshape(T, m.HV, m.d),
        beta=host(s["beta"]), g=host(s["g"]), per_channel=per_channel, pool=pool64)
    assert rel(host(s["o"]), o_ref) <= 2e-3
    o, gate = host(s["o"]), host(s["gate"]).reshape(T, m.HV, m.d)
    n = ol.rms(o, 1e-6)[0]
    check("z", s["z"], ol.gated_norm(o, gate, host(m.out_w), "silu"), 96 * U * np.abs(n * host(m.out_w) * gate))
    z = host(s["z"]).reshape(T, N)
    ref = ol.linear(z, host(m.w_o), None, "none", host(s["h"]))[0]
    check("out", s["out"], ref, product_tol(z, host(m.w_o).T, N, "bf16") + 4 * U * np.abs(ref))


def test_layer_decode_follows_prefill():
    """Tokens fed one at a time (the single-token forms of every operator) give what one prefill of
    the same tokens gives.  Prefill and decode each stay within 2e-3 of the recurrence (relative
    to the largest output), the output norm and projection keep relative sizes, and the bf16
    roundings of both runs (front end, z) may differ by a step of 2^-7: 1.2e-2 in all, of the
    projection's part of the output."""
    B, steps = 5, 6
    m = Model(3)
    r = rng(4)
    T, N, CD = B * steps, m.HV * m.d, m.w_in.shape[0]
    block, _ = dev(r.standard_normal((T, N)), "bf16")
    stream, _ = dev(r.standard_normal((T, N)), "f32")
    conv0, _ = dev(r.standard_normal((B + 1, CD, 3)), "bf16")
    pool0, _ = dev(r.standard_normal((B + 1, m.HV, m.d, m.d)) * 0.02, "f32")
    slots = i32(np.arange(B)[::-1].copy())
    off = i32(np.arange(B + 1) * steps)
    whole = m.run(block, stream, conv0.clone(), pool0.clone(), slots, off)
    conv, pool = conv0.clone(), pool0.clone()
    outs = []
    for t in range(steps):
        rows = torch.arange(B, device=DEV) * steps + t
        s = m.run(block[rows].contiguous(), stream[rows].contiguous(), conv, pool, slots)
        outs.append(s["out"] - s["h"])
    no_error()
    got = host(torch.stack(outs, 1).reshape(T, N))
    ref = host(whole["out"] - whole["h"])
    assert rel(got, ref) <= 1.2e-2


def test_layer_gradients_reach_the_recurrence():
    """The gradient of the layer's output goes back through the output projection and norm into
    prefill_bwd: each stage against the reference on what it was given."""
    p = workloads.make_problem("layer", num_seqs=3, lengths=[70, 1, 130], num_k_heads=2,
                               num_v_heads=4, d=128, qkv_dtype="bf16", state_dtype="f32",
                               decay_kind="per_channel", chunk=64, zero_state=False, seed=5)
    t = torch_io.prefill_inputs(p, DEV)
    pool0 = t["state_pool"].clone()
    r = rng(6)
    T, HV, d = p.total_tokens, 4, 128
    N = HV * d
    gate, gate64 = dev(r.standard_normal((T, HV, d)), "bf16")
    nw, nw64 = dev(1 + 0.1 * r.standard_normal(d), "f32")
    wo, wo64 = dev(r.standard_normal((N, N)) / np.sqrt(N), "bf16")
    d_out, d_out64 = dev(r.standard_normal((T, N)), "bf16")
    o = kda.prefill(**t, chunk=64)
    z = kda.gated_norm(o, gate, nw, activation="silu")
    dz, dwo, _ = kda.linear_bwd(z.view(T, N), wo, d_out)
    d_o, d_gate, d_nw = kda.gated_norm_bwd(o, gate, nw, dz.view(T, HV, d), activation="silu")
    grads = kda.prefill_bwd(t["q"], t["k"], t["v"], t["beta"], t["log_decay"], t["input_row_offsets"],
                            t["slot_idx"], pool0, d_o, None, chunk=64)
    no_error()
    z64 = host(z).reshape(T, N)
    dz_ref, dwo_ref, _, _ = ol.linear_bwd(z64, wo64, d_out64)
    check("dz", dz, dz_ref, product_tol(d_out64, wo64, N, "bf16") + 2 * U * np.abs(dz_ref))
    check("dwo", dwo, dwo_ref, product_tol(d_out64.T, z64, T, "bf16") + 2 * U * np.abs(dwo_ref))
    o64, dz64 = host(o), host(dz).reshape(T, HV, d)
    n, rr = ol.rms(o64, 1e-6)
    a = np.abs(ol.act("silu", gate64)) + 1e-30
    dn = np.abs(dz64) * np.maximum(a, np.abs(gate64)) * np.abs(nw64)
    ro, rg, rw = ol.gated_norm_bwd(o64, gate64, nw64, dz64, "silu")
    check("d_o", d_o, ro, 256 * U * rr * (dn + np.abs(n) * np.mean(dn * np.abs(n), -1, keepdims=True)))
    check("d_gate", d_gate, rg, 128 * U * np.abs(dz64 * n * nw64) * (1 + np.abs(gate64)))
    check("d_weight", d_nw, rw, (T * HV + 256) * U * (dn / np.abs(nw64) * np.abs(n)).reshape(-1, d).sum(0))
    ref = oracle.backward(p, host(d_o), None)
    for name, g in zip(("dq", "dk", "dv", "dbeta", "dg", "d_state0"), grads):
        assert rel(host(g), ref[name]) <= 2e-3, name


# --------------------------------------------------------------------------- how calls are launched

def operands(T, K, N, seed=0, dtype="bf16"):
    r = rng(20, seed, T, K, N)
    t = dict(x=dev(r.standard_normal((T, K)), dtype)[0], w=dev(r.standard_normal((N, K)), dtype)[0],
             b=dev(r.standard_normal(N), "f32")[0], dy=dev(r.standard_normal((T, N)), dtype)[0],
             o=dev(r.standard_normal((T, 2, 64)), "f32")[0], og=dev(r.standard_normal((T, 2, 64)), "bf16")[0],
             nw=dev(r.standard_normal(64), "f32")[0], kw=dev(r.standard_normal(K), "f32")[0])
    t["ody"] = t["og"].flip(0).contiguous()
    return t


def everything(t):
    """Every entry point once, on one set of operands."""
    y, z = kda.linear(t["x"], t["w"], t["b"], activation="silu", save_pre_activation=True)
    out = [y, z]
    out += kda.linear_bwd(t["x"], t["w"], t["dy"], activation="silu", pre_activation=z, need_bias=True)
    n, h = kda.residual_norm(t["x"], t["kw"], residual=t["x"], post_weight=t["kw"], gate=t["kw"])
    out += [n, h]
    out += kda.residual_norm_bwd(t["x"], h, t["kw"], t["x"], h, post_weight=t["kw"], gate=t["kw"])
    out.append(kda.gated_norm(t["o"], t["og"], t["nw"]))
    out += kda.gated_norm_bwd(t["o"], t["og"], t["nw"], t["ody"])
    return out


SHAPES = [(1, 256, 64), (33, 264, 100), (1700, 512, 1600)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_replays_on_new_inputs(T, K, N, dtype):
    """Captured once, replayed on other contents of the same buffers: the same bits as eager calls."""
    t = operands(T, K, N, 0, dtype)
    everything(t)                                            # warm-up outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = everything(t)
    for seed in (1, 2):
        new = operands(T, K, N, seed, dtype)
        for k in t:
            t[k].copy_(new[k])
        g.replay()
        eager = everything(new)
        no_error()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_two_graphs_interleaved():
    """Two graphs, each with the workspaces of its own capture, replayed in turns and at once."""
    ts = [operands(300, 256, 200, s) for s in (3, 4)]
    graphs, outs, refs = [], [], []
    for t in ts:
        refs.append([a.clone() for a in everything(t)])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(t))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    no_error()
    for o, r in zip(outs, refs):
        assert all(torch.equal(a, b) for a, b in zip(o, r))


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_streams_at_once(T, K, N):
    """Calls on several streams at once, by `stream=` and by the current stream."""
    ts = [operands(T, K, N, s) for s in range(3)]
    refs = [[a.clone() for a in everything(t)] for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    outs = []
    for t, s in zip(ts, streams):
        with torch.cuda.stream(s):
            outs.append(everything(t))
    named = [kda.linear(t["x"], t["w"], stream=s) for t, s in zip(ts, streams)]
    no_error()
    for o, r in zip(outs, refs):
        assert all(torch.equal(a, b) for a, b in zip(o, r))
    for t, y in zip(ts, named):
        assert torch.equal(y, kda.linear(t["x"], t["w"]))


def canary(nbytes):
    """A workspace of exactly nbytes between guards, everything 0xff (NaN as a float)."""
    buf = torch.full((nbytes + 512,), 255, dtype=torch.uint8, device=DEV)
    return buf, buf[256:256 + nbytes]


def intact(buf):
    assert (buf[:256] == 255).all() and (buf[-256:] == 255).all()


@pytest.mark.parametrize("T,K,N", [(5, 100, 37), (33, 264, 101), (300, 200, 600)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspace_stays_within_its_size(T, K, N, dtype):
    """Workspaces of exactly the size asked for, full of NaN on entry: the same results, and nothing
    written outside."""
    t = operands(T, K, N, 5, dtype)
    z = torch.empty((T, N), dtype=t["x"].dtype, device=DEV).normal_()

    def calls(ws):
        yield "linear", lambda w: kda.linear(t["x"], t["w"], t["b"], workspace=w)
        yield "linear_bwd", lambda w: kda.linear_bwd(t["x"], t["w"], t["dy"], activation="gelu",
                                                     pre_activation=z, need_bias=True, workspace=w)
        yield "residual_norm_bwd", lambda w: kda.residual_norm_bwd(
            t["x"], t["x"], t["kw"], t["x"], post_weight=t["kw"], gate=t["kw"], workspace=w)
        yield "gated_norm_bwd", lambda w: kda.gated_norm_bwd(t["o"], t["og"], t["nw"], t["ody"], workspace=w)
    for name, call in calls(None):
        layer._PLANS.clear()
        plain = call(None)
        (plan,) = layer._PLANS.values()
        buf, ws = canary(plan.nbytes)
        again = call(ws if plan.nbytes else None)
        no_error()
        intact(buf)
        for a, b in zip(plain if isinstance(plain, tuple) else [plain],
                        again if isinstance(again, tuple) else [again]):
            assert (a is None and b is None) or torch.equal(a, b), name
        if plan.nbytes:
            with pytest.raises(ValueError, match="workspace"):
                call(ws[:-1])


def test_outputs_stay_within_their_rows():
    """y, z, dx and dw end at ragged edges of every tile size: guards behind them stay."""
    for T, K, N in [(129, 72, 130), (70, 136, 264), (1601, 264, 1539)]:
        t = operands(T, K, N, 6)
        out = torch.full((T + 3, N + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        kda.linear(t["x"], t["w"], out=out[:T, :N])
        no_error()
        assert (out[T:] == 7).all() and (out[:T, N:] == 7).all()
        assert torch.equal(out[:T, :N], kda.linear(t["x"], t["w"]))


def test_device_error_word_stays_clear_and_status_raises():
    t = operands(33, 264, 100, 7)
    everything(t)
    no_error()
    p = layer._linear_params(t["x"], t["w"], "none", 1.0, torch.bfloat16, 0)
    st = _lib.load().kda_linear_fwd(ctypes.byref(p), None, None, None, None, None, None, None, 0, None)
    assert st == _lib.KDA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        kda.linear(t["x"], t["w"], residual=t["x"])
    with pytest.raises(ValueError):
        kda.linear(t["x"], t["w"].cpu())
    with pytest.raises(kda.KdaError):
        kda.residual_norm(t["x"], t["kw"], eps=0.0)


def test_scalars_given_as_tensors_are_read_each_call():
    """A scale or eps held in a tensor that changes between calls: as with the numbers themselves."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn(5, 64, generator=g).to(DEV)
    w = torch.randn(48, 64, generator=g).to(DEV)
    kw = torch.randn(64, generator=g).to(DEV)
    s, eps = torch.tensor(0.5), torch.tensor(1e-6)
    for a, e in [(0.5, 2.0 ** -20), (2.0, 0.25)]:
        s.fill_(a)
        eps.fill_(e)
        y = kda.linear(x, w, scale=a)
        assert torch.equal(kda.linear(x, w, scale=s), y)
        for got, want in zip(kda.linear_bwd(x, w, y, scale=s), kda.linear_bwd(x, w, y, scale=a)):
            assert got is want or torch.equal(got, want)
        n, h = kda.residual_norm(x, kw, scale=a, eps=e)
        for got, want in zip(kda.residual_norm(x, kw, scale=s, eps=eps), (n, h)):
            assert torch.equal(got, want)
        for got, want in zip(kda.residual_norm_bwd(x, h, kw, n, scale=s, eps=eps),
                             kda.residual_norm_bwd(x, h, kw, n, scale=a, eps=e)):
            assert got is want or torch.equal(got, want)
        o = x.view(5, 2, 32)
        v = kda.gated_norm(o, o, kw[:32], eps=e)
        assert torch.equal(kda.gated_norm(o, o, kw[:32], eps=eps), v)
        for got, want in zip(kda.gated_norm_bwd(o, o, kw[:32], v, eps=eps),
                             kda.gated_norm_bwd(o, o, kw[:32], v, eps=e)):
            assert torch.equal(got, want)
    no_error()
