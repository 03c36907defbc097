"""The short convolution on the GPU against its float64 definition (oracle/layer_oracle.py).

Tolerances count roundings, u = 2^-24 for one in fp32, half a step of the output's type for
the store.  The sum of W products and the bias is off by at most (W + 2) u times the sum of its
terms' sizes.  SiLU multiplies an error of its argument by at most 1.1, and adds its own: the
exponent's argument, rounded, is off by |x| u, its power of two, the sum and the reciprocal by
4 u each, so (|x| + 16) u of the result.  dL/dpre = dy SiLU'(pre) with |SiLU'| <= 1.1 and
|SiLU''| <= 0.5; its terms s and x s (1 - s) are each off by (|x| + 24) u.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_log2_amd as kda
from oracle import layer_oracle as lo

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# (type, B, T, D, W, SiLU, bias, offsets, initial state, token stride beyond D)
CASES = {
    "one token": ("bf16", 1, 1, 64, 4, True, True, None, True, 0),
    "one token without a state": ("fp32", 3, 1, 8, 2, False, False, None, False, 0),
    "shorter than the window": ("bf16", 2, 2, 40, 4, True, False, None, True, 0),
    "channels not in eights": ("bf16", 2, 37, 83, 3, True, True, None, True, 0),
    "one channel": ("fp32", 1, 9, 1, 4, True, True, None, True, 0),
    "seven channels": ("bf16", 1, 33, 7, 4, True, True, None, False, 0),
    "several workgroups": ("bf16", 1, 531, 600, 4, True, True, None, True, 0),
    "in 32 bits": ("fp32", 2, 203, 130, 4, True, True, None, True, 0),
    "width two": ("fp32", 1, 65, 512, 2, False, True, None, True, 0),
    "a slice of a projection": ("bf16", 2, 50, 96, 4, True, True, None, True, 32),
    "an odd slice": ("bf16", 1, 70, 45, 3, False, True, None, True, 6),
    "packed": ("bf16", 1, 200, 72, 4, True, True, [0, 0, 1, 3, 60, 61, 127, 200, 200], True, 0),
    "packed without states": ("fp32", 1, 150, 24, 3, True, False, [0, 2, 2, 4, 149, 150], False, 0),
    "one packed sequence": ("bf16", 1, 77, 16, 4, False, True, [0, 77], True, 8),
    "all empty": ("bf16", 1, 0, 16, 4, True, True, [0, 0, 0], True, 0),
}


def make(case, seed=0):
    kind, B, T, D, W, silu, bias, cu, state, extra = CASES[case]
    g = torch.Generator().manual_seed(seed)
    t = TYPES[kind]
    n = B if cu is None else len(cu) - 1
    x = torch.randn(B, T, D + extra, generator=g).to(t)[..., extra // 2:extra // 2 + D]
    a = dict(x=x, weight=torch.randn(D, W, generator=g) / 2, bias=torch.randn(D, generator=g) if bias else None,
             h0=torch.randn(n, W - 1, D, generator=g).to(t) if state else None,
             dy=torch.randn(B, T, D, generator=g).to(t), dht=torch.randn(n, W - 1, D, generator=g).to(t))
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int64)
    return a, cu_t, silu, t


def on_gpu(v):
    if v is None:
        return None
    if v.is_contiguous():
        return v.to(DEV)
    wide = torch.empty(v.shape[:-1] + (v.stride(-2),), dtype=v.dtype, device=DEV)  # keep the view's strides
    off = v.storage_offset()
    wide[..., off:off + v.shape[-1]] = v.to(DEV)
    return wide[..., off:off + v.shape[-1]]


def forward(a, cu, silu):
    d = {k: on_gpu(v) for k, v in a.items()}
    return d, kda.short_conv(d["x"], d["weight"], d["bias"], "silu" if silu else None, d["h0"], True,
                             None if cu is None else cu.to(DEV), cu_seqlens_host=cu)


def check(name, got, want, bound):
    off = (got.double().cpu() - want).abs()
    worst = (off / bound.clamp(min=1e-300)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    a, cu, silu, t = make(case)
    _, (y, ht) = forward(a, cu, silu)
    want, last, pre, size = lo.short_conv(a["x"], a["weight"], a["bias"], silu, a["h0"], cu)
    W = a["weight"].shape[1]
    bound = torch.finfo(t).eps / 2 * want.abs() + 1.1 * (W + 2) * U * size + (pre.abs() + 16) * U * want.abs() + 1e-30
    check("y", y, want, bound)
    assert torch.equal(ht.double().cpu(), last)  # inputs, unchanged


def bwd_bounds(a, cu, silu, t, want, sizes, pre, size):
    """Bounds of every gradient: an error E of each dL/dpre, carried through the sums."""
    W = a["weight"].shape[1]
    dy = a["dy"].double().abs()
    E = dy * ((0.5 * (W + 2) * size + 2 * (pre.abs() + 24) * (1 + pre.abs())) * U if silu else 0)
    through, _ = lo.short_conv_bwd(a["x"], a["weight"].abs(), E, None, False, a["h0"], None, cu)
    half, n = torch.finfo(t).eps / 2, a["x"].shape[0] * a["x"].shape[1]
    depth = 32 + 256 + n / 128 + W  # a run's sum, the workgroup's runs, the workgroups
    xs = a["x"].double().abs()
    hs = None if a["h0"] is None else a["h0"].double().abs()
    sums, _ = lo.short_conv_bwd(xs, a["weight"], E, None, False, hs, None, cu)
    return dict(dx=half * want["dx"].abs() + (W + 3) * U * sizes["dx"] + through["dx"] + 1e-30,
                dh0=half * want["dh0"].abs() + (W + 3) * U * sizes["dh0"] + through["dh0"] + 1e-30,
                dweight=depth * U * sizes["dweight"] + sums["dweight"] + 1e-30,
                dbias=depth * U * sizes["dbias"] + E.sum((0, 1)) + 1e-30)


def backward(d, cu, silu, dy):
    return kda.short_conv_bwd(d["x"], d["weight"], dy, d["bias"], "silu" if silu else None, d["h0"], d["dht"],
                              None if cu is None else cu.to(DEV), cu_seqlens_host=cu)


@pytest.mark.gpu
@pytest.mark.parametrize("wide_dy", [False, True], ids=["dy as x", "dy in 32 bits"])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, wide_dy):
    a, cu, silu, t = make(case, 1)
    d = {k: on_gpu(v) for k, v in a.items()}
    got = backward(d, cu, silu, d["dy"].float() if wide_dy else d["dy"])
    _, _, pre, size = lo.short_conv(a["x"], a["weight"], a["bias"], silu, a["h0"], cu)
    want, sizes = lo.short_conv_bwd(a["x"], a["weight"], a["dy"], a["bias"], silu, a["h0"], a["dht"], cu)
    bounds = bwd_bounds(a, cu, silu, t, want, sizes, pre, size)
    assert set(got) == {"dx", "dweight"} | ({"dbias"} if a["bias"] is not None else set()) | ({"dh0"} if a["h0"] is not None else set())
    for k, v in got.items():
        assert v.dtype == (t if k in ("dx", "dh0") else torch.float32)
        check(k, v, want[k], bounds[k])


@pytest.mark.gpu
def test_sequences_of_a_pack_alone():
    """A sequence in a pack and by itself: the same bits, forward and dx."""
    a, cu, silu, _ = make("packed", 3)
    d, (y, ht) = forward(a, cu, silu)
    grads = backward(d, cu, silu, d["dy"])
    for n, (p, q) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        if p == q:
            continue
        one = dict(d, x=d["x"][:, p:q].contiguous(), h0=d["h0"][n:n + 1], dht=d["dht"][n:n + 1])
        y1, h1 = kda.short_conv(one["x"], one["weight"], one["bias"], "silu", one["h0"], True)
        assert torch.equal(y1, y[:, p:q]) and torch.equal(h1, ht[n:n + 1])
        g1 = backward(one, None, silu, d["dy"][:, p:q].contiguous())
        assert torch.equal(g1["dx"], grads["dx"][:, p:q]) and torch.equal(g1["dh0"], grads["dh0"][n:n + 1])


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_windows():
    x = torch.randn(1, 40, 16, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    w = torch.full((16, 4), 0.5)
    clean, _ = kda.short_conv(x.to(DEV), w.to(DEV), activation="silu")
    bad = x.clone()
    bad[0, 10, 3], bad[0, 20, 5] = float("nan"), float("inf")
    y, _ = kda.short_conv(bad.to(DEV), w.to(DEV), activation="silu")
    same = torch.ones(1, 40, 16, dtype=torch.bool, device=DEV)
    same[0, 10:14, 3] = same[0, 20:24, 5] = False
    assert torch.equal(y[same], clean[same])
    assert y[0, 10:14, 3].isnan().all() and y[0, 20:24, 5].isinf().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D,W,silu,extra", [(64, 4, True, 0), (301, 3, True, 5), (8, 2, False, 0)])
def test_step(kind, D, W, silu, extra):
    t, g = TYPES[kind], torch.Generator().manual_seed(4)
    rows, pool = 9, 13
    x = torch.randn(rows, D + extra, generator=g).to(t)[:, :D]
    state = torch.randn(pool, W - 1, D, generator=g).to(t)
    weight, bias = torch.randn(D, W, generator=g) / 2, torch.randn(D, generator=g)
    slots = torch.tensor([5, 0, 12, -1, 3, 7, 13, 1, 2], dtype=torch.int32)
    dev_state = state.to(DEV)
    wide = torch.zeros(rows, D + extra, dtype=t, device=DEV)
    wide[:, :D] = x.to(DEV)
    y = kda.short_conv_step(wide[:, :D], dev_state, weight.to(DEV), bias.to(DEV), "silu" if silu else None, slots.to(DEV))
    expect = state.clone()
    for r, s in enumerate(slots.tolist()):
        if not 0 <= s < pool:
            assert (y[r] == 0).all()
            continue
        want, last, pre, size = lo.short_conv(x[r][None, None], weight, bias, silu, state[s][None])
        bound = torch.finfo(t).eps / 2 * want.abs() + 1.1 * (W + 2) * U * size + (pre.abs() + 16) * U * want.abs() + 1e-30
        check("y", y[r], want[0, 0], bound[0, 0])
        expect[s] = last[0].to(t)
    assert torch.equal(dev_state.cpu(), expect)


@pytest.mark.gpu
def test_steps_continue_a_prompt():
    """A prompt and then single tokens: what the whole sequence gives at once, to its roundings."""
    a, _, silu, t = make("several workgroups", 6)
    d = {k: on_gpu(v) for k, v in a.items()}
    whole, last = kda.short_conv(d["x"], d["weight"], d["bias"], "silu", d["h0"], True)
    y, state = kda.short_conv(d["x"][:, :500].contiguous(), d["weight"], d["bias"], "silu", d["h0"], True)
    steps = [kda.short_conv_step(d["x"][:, i], state, d["weight"], d["bias"], "silu") for i in range(500, 531)]
    assert torch.equal(y, whole[:, :500]) and torch.equal(state, last)
    tail, want = torch.stack(steps, 1).double(), whole[:, 500:].double()
    assert ((tail - want).abs() <= torch.finfo(t).eps * want.abs() + 1e-6).all()


@pytest.mark.gpu
def test_captured_and_replayed():
    a, cu, silu, _ = make("packed", 8)
    d = {k: on_gpu(v) for k, v in a.items()}
    cu_dev = cu.to(DEV)
    state = d["h0"].clone()

    def everything():
        y, ht = kda.short_conv(d["x"], d["weight"], d["bias"], "silu", d["h0"], True, cu_dev, cu_seqlens_host=cu)
        g = kda.short_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], "silu", d["h0"], d["dht"], cu_dev, cu_seqlens_host=cu)
        s = kda.short_conv_step(d["x"][0, :len(state)], state, d["weight"], d["bias"], "silu")
        return [y, ht, s, *g.values()]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything()
    for seed in range(3):
        d["x"].copy_(torch.randn(d["x"].shape, generator=torch.Generator().manual_seed(seed)))
        state.copy_(d["h0"])
        graph.replay()
        torch.cuda.synchronize()
        got, moved = [v.clone() for v in out], state.clone()
        state.copy_(d["h0"])
        for x, y in zip(got, everything()):
            assert torch.equal(x, y)
        assert torch.equal(moved, state)


@pytest.mark.gpu
def test_another_stream():
    a, cu, silu, _ = make("several workgroups", 9)
    d, (y, ht) = forward(a, cu, silu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, ht2 = kda.short_conv(d["x"], d["weight"], d["bias"], "silu", d["h0"], True)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(ht, ht2)


@pytest.mark.gpu
def test_refusals_on_the_device():
    x, w = torch.zeros(2, 6, 16, device=DEV), torch.zeros(16, 4, device=DEV)
    bad = [
        lambda: kda.short_conv(x.transpose(0, 1), w), lambda: kda.short_conv(x[:, :, ::2], w[:8]),
        lambda: kda.short_conv(x[:, ::2][:, :2], w, initial_state=torch.zeros(1, 3, 16, device=DEV)),
        lambda: kda.short_conv(x.double(), w), lambda: kda.short_conv(x, w.half()), lambda: kda.short_conv(x, w, activation="gelu"),
        lambda: kda.short_conv(x, w, cu_seqlens=torch.tensor([0, 6])), lambda: kda.short_conv(x, w, w[:, 0].cpu()),
        lambda: kda.short_conv(x[:1].expand(2, 6, 16), w),
        lambda: kda.short_conv_bwd(x, w, x.bfloat16()), lambda: kda.short_conv_bwd(x, w, x[:, :5]),
        lambda: kda.short_conv_step(x[:, 0], x[:, :3].contiguous(), w, slots=torch.zeros(2, dtype=torch.int64, device=DEV)),
        lambda: kda.short_conv_step(x[:, 0], x[:1, :3].contiguous(), w),
    ]
    for f in bad:
        with pytest.raises(kda.KDAContractError):
            f()
