"""The state space scan on the GPU against its float64 definition (oracle/layer_oracle.py).

Bounds.  Run on the absolute values of x, B, C, dy and the states, the definition gives for each
output the sum of the sizes of its terms (every sum then has terms of one sign); an error bound is
a number of roundings relative to that.  u = 2^-24 is a rounding in fp32, h half a step of the
inputs' type (2^-8 for bf16; u for fp32).  With
  c = N + P + 2 L + 64 + 2 (chunks): the longest chains of fp32 additions of a product, a chunk's
      tokens, the chunks' states, and the decays' own roundings, (|exponent| + 2) u with a weight
      of e^-|exponent|;
states and their gradients are off by c u of their sizes (for bf16 inputs too, whose scaled x or dy
goes through the products in three parts, 24 bits).  y, dx, dB and dC pass through one
more rounding of a product's operand and one at the store: h of their size, and h of themselves.
The decays' gradients are differences: sums over the rest of a chunk of dy . (y - D x) minus sums of
the parts with both tokens behind t, so their errors are relative to twice that sum besides the size
of the result.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_log2_amd as kda
from oracle import layer_oracle as lo

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# type, B, T, H, G, N, P, offsets, softplus, with D / dt_bias / states, tokens' extra stride
CASES = {
    "one token": ("bf16", 1, 1, 2, 1, 32, 32, None, True, True, 0),
    "one token without states": ("fp32", 3, 1, 1, 1, 32, 64, None, False, False, 0),
    "a chunk less one": ("bf16", 1, 63, 2, 2, 64, 64, None, True, True, 0),
    "a chunk": ("bf16", 2, 64, 2, 1, 128, 64, None, True, True, 0),
    "a chunk and one": ("bf16", 1, 65, 4, 2, 128, 128, None, True, True, 0),
    "a chunk and one in 32 bits": ("fp32", 1, 33, 3, 1, 128, 128, None, True, True, 0),
    "odd tiles": ("bf16", 1, 150, 3, 1, 96, 96, None, True, True, 0),
    "odd tiles in 32 bits": ("fp32", 1, 100, 3, 3, 96, 32, None, True, True, 0),
    "small state": ("bf16", 2, 97, 6, 2, 32, 64, None, True, False, 0),
    "wide heads": ("bf16", 1, 130, 4, 1, 32, 128, None, False, True, 0),
    "tall state": ("fp32", 1, 70, 2, 1, 128, 32, None, True, True, 0),
    "one group": ("bf16", 1, 90, 8, 1, 64, 32, None, True, True, 0),
    "slices of a projection": ("bf16", 2, 77, 4, 2, 64, 64, None, True, True, 24),
    "odd slices": ("bf16", 1, 77, 2, 1, 32, 32, None, True, True, 5),
    "slices in 32 bits": ("fp32", 2, 40, 2, 2, 64, 32, None, True, True, 3),
    "segments": ("bf16", 1, 700, 2, 1, 64, 64, None, True, True, 0),
    "segments in 32 bits": ("fp32", 2, 300, 2, 1, 32, 32, None, True, True, 0),
    "packed": ("bf16", 1, 420, 4, 2, 64, 64, [0, 0, 1, 64, 129, 130, 420, 420], True, True, 0),
    "packed in 32 bits": ("fp32", 1, 230, 2, 1, 64, 96, [0, 200, 200, 231 - 1], True, True, 0),
    "packed without states": ("bf16", 1, 300, 2, 1, 32, 64, [0, 290, 300], True, False, 0),
    # batches that fill the GPU uncut, a segment to a sequence of several chunks
    "whole sequences": ("bf16", 40, 200, 16, 4, 32, 32, None, True, True, 0),
    "whole sequences in 32 bits": ("fp32", 24, 100, 32, 8, 32, 32, None, True, True, 0),
    "one long sequence among short ones": ("bf16", 1, 2260, 32, 8, 32, 64, [0, *range(700, 2261, 130)], True, True, 0),
    "pairs of heads in 32 bits": ("fp32", 2, 100, 4, 1, 128, 64, None, True, True, 0),
    "all empty": ("bf16", 1, 0, 2, 1, 32, 32, [0, 0, 0], True, True, 0),
}


def strided(v, extra, g):
    """v as a view whose tokens lie `extra` elements further apart."""
    if not extra or v.numel() == 0:
        return v
    flat = v.flatten(2)
    return torch.zeros(*flat.shape[:2], flat.shape[2] + extra, dtype=v.dtype)[..., extra // 2:extra // 2 + flat.shape[2]].copy_(flat).unflatten(2, v.shape[2:])


def make(case, seed=0, strong=False):
    kind, nb, T, H, G, N, P, cu, softplus, more, extra = CASES[case]
    g = torch.Generator().manual_seed(seed)
    t = TYPES[kind]
    n = nb if cu is None else len(cu) - 1

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g) * std

    a = dict(x=normal(nb, T, H, P).to(t), dt=(normal(nb, T, H) if softplus else torch.rand(nb, T, H, generator=g) * 0.2).to(t),
             A_log=torch.rand(H, generator=g) * 2.8, B=normal(nb, T, G, N, std=N ** -0.25).to(t),
             C=normal(nb, T, G, N, std=N ** -0.25).to(t), D=normal(H) if more else None,
             dt_bias=(normal(H) + (4.0 if strong else -3.0) if more and softplus else None),
             h0=normal(n, H, N, P, std=0.3) if more else None)
    for k in ("x", "dt", "B", "C"):
        a[k] = strided(a[k], extra, g)
    grads = dict(dy=normal(nb, T, H, P).to(t), dht=normal(n, H, N, P, std=0.3))
    return a, grads, None if cu is None else torch.tensor(cu, dtype=torch.int64), softplus, t


def on_gpu(v):
    if v is None or v.is_contiguous():
        return None if v is None else v.to(DEV)
    last = v.storage_offset() + sum((n - 1) * step for n, step in zip(v.shape, v.stride()))
    base = torch.zeros(last + 1, dtype=v.dtype, device=DEV)
    return base.as_strided(v.shape, v.stride(), v.storage_offset()).copy_(v.to(DEV))


def forward(a, cu, softplus):
    d = {k: on_gpu(v) for k, v in a.items()}
    return d, kda.chunk_ssm(d["x"], d["dt"], d["A_log"], d["B"], d["C"], d["D"], d["dt_bias"], softplus, d["h0"], True,
                            None if cu is None else cu.to(DEV), cu_seqlens_host=cu)


def backward(d, grads, cu, softplus):
    return kda.chunk_ssm_bwd(d["x"], d["dt"], d["A_log"], d["B"], d["C"], grads["dy"].to(DEV), grads["dht"].to(DEV), d["D"],
                             d["dt_bias"], softplus, d["h0"], None if cu is None else cu.to(DEV), cu_seqlens_host=cu)


def constants(a, t):
    N, P, T = a["B"].shape[3], a["x"].shape[3], a["x"].shape[1]
    L = 64 if t == torch.bfloat16 else 32
    c = (N + P + 2 * L + 64 + 2 * (T // L + 1)) * U
    return (torch.finfo(t).eps / 2 if t == torch.bfloat16 else U), c


def sizes_of(a):
    """The inputs' absolute values (without D's term, whose rounding is its own)."""
    return {k: None if a[k] is None else a[k].abs() if k in ("x", "B", "C", "h0") else a[k] for k in a}


def check(name, got, want, bound):
    assert got.shape == want.shape
    off = (got.double().cpu() - want).abs()
    worst = (off / (bound + 1e-30)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound"


def near(name, got, want, t, state=False):
    """Over many values independent roundings add up as their squares: the root mean square of a
    rounding is at most h / sqrt 3.  Three of them (operand, state, store) are h together; states,
    and every value in fp32, have chains' sqrt c u, 1.5e-6 for the c of at most 600 here."""
    if want.numel() > 2000:
        rel = ((got.double().cpu() - want).norm() / want.norm()).item()
        h = 2.0 ** -8 if t == torch.bfloat16 else 0.0
        assert rel <= (0.0 if state else h) + 1.5e-6, f"{name}: {rel:.3g} in the norm"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("strong", [False, True], ids=["slow", "fast"])
def test_forward(case, strong):
    a, _, cu, softplus, t = make(case, strong=strong)
    _, (y, ht) = forward(a, cu, softplus)
    want, last = lo.ssm(a["x"], a["dt"], a["A_log"], a["B"], a["C"], a["D"], a["dt_bias"], softplus, a["h0"], cu)
    z = sizes_of(a)
    size, size_last = lo.ssm(z["x"], z["dt"], z["A_log"], z["B"], z["C"], None, z["dt_bias"], softplus, z["h0"], cu)
    h, s = constants(a, t)
    skip = 0 if a["D"] is None else 4 * U * (a["D"].double()[:, None] * a["x"].double()).abs()
    check("y", y, want, h * want.abs() + (h + s) * size + skip)
    check("final state", ht, last, s * size_last)
    near("y", y, want, t)
    near("final state", ht, last, t, True)
    assert y.dtype == t and ht.dtype == torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("strong", [False, True], ids=["slow", "fast"])
def test_backward(case, strong):
    a, grads, cu, softplus, t = make(case, 1, strong)
    d = {k: on_gpu(v) for k, v in a.items()}
    got = backward(d, grads, cu, softplus)
    args = (a["dt_bias"], softplus)
    want = lo.ssm_bwd(a["x"], a["dt"], a["A_log"], a["B"], a["C"], grads["dy"], grads["dht"], a["D"], *args, a["h0"], cu)
    z = sizes_of(a)
    dy, dht = grads["dy"].abs(), grads["dht"].abs()
    size = lo.ssm_bwd(z["x"], z["dt"], z["A_log"], z["B"], z["C"], dy, dht, None, *args, z["h0"], cu)
    y_size, _ = lo.ssm(z["x"], z["dt"], z["A_log"], z["B"], z["C"], None, *args, z["h0"], cu)
    h, s = constants(a, t)
    group = a["x"].shape[2] // a["B"].shape[2]
    bounds = {k: h * want[k].abs() + (h + s + group * U) * size[k] for k in ("dB", "dC")}
    skip = 0 if a["D"] is None else 4 * U * (a["D"].double()[:, None] * grads["dy"].double()).abs()
    bounds["dx"] = h * want["dx"].abs() + (h + s) * size["dx"] + skip
    bounds["dh0"] = s * size["dh0"]
    # the rest of each chunk: at most 64 tokens from t on, of any sequence
    rows = (y_size * dy.double()).sum(-1)
    rest = rows.clone()
    for k in range(1, 64):
        rest[:, :rows.shape[1] - k] += rows[:, k:] if k < rows.shape[1] else 0
    dl = (s + 64 * U) * (2 * rest + size["dl"])
    A, steps = torch.exp(a["A_log"].double()), lo.ssm_steps(a["dt"], *args)[0].abs()
    dd = A * dl + (s + 8 * U) * size["direct"] + 8 * U * A * want["dl"].abs()
    n = a["x"].shape[0] * a["x"].shape[1]
    bounds["ddt"] = torch.finfo(a["dt"].dtype).eps / 2 * want["ddt"].abs() + dd
    total = (n / 256 + 80) * U
    bounds["ddt_bias"] = dd.sum((0, 1)) + total * want["ddt"].abs().sum((0, 1))
    bounds["dA_log"] = (dl * steps * A).sum((0, 1)) + (total + 4 * U) * (want["dl"] * steps * A).abs().sum((0, 1))
    bounds["dD"] = (s + total) * (dy.double() * z["x"].double()).sum((0, 1, 3))
    names = {"dx", "ddt", "dA_log", "dB", "dC"} | {n for n, k in (("dD", "D"), ("ddt_bias", "dt_bias"), ("dh0", "h0")) if a[k] is not None}
    assert set(got) == names
    for k, v in got.items():
        check(k, v, want[k], bounds[k])
        if k in ("dx", "dB", "dC"):
            near(k, v, want[k], t)
        assert v.dtype == (t if k in ("dx", "dB", "dC", "ddt") else torch.float32)


@pytest.mark.gpu
def test_steps_in_32_bits_beside_bf16():
    a, grads, cu, softplus, t = make("a chunk and one", 2)
    a["dt"] = a["dt"].float() * 1.001
    d, (y, ht) = forward(a, cu, softplus)
    want, last = lo.ssm(a["x"], a["dt"], a["A_log"], a["B"], a["C"], a["D"], a["dt_bias"], softplus, a["h0"])
    near("y", y, want, t)
    near("final state", ht, last, t, True)
    got = backward(d, grads, cu, softplus)
    full = lo.ssm_bwd(a["x"], a["dt"], a["A_log"], a["B"], a["C"], grads["dy"], grads["dht"], a["D"], a["dt_bias"], softplus, a["h0"])
    assert got["ddt"].dtype == torch.float32
    rel = ((got["ddt"].double().cpu() - full["ddt"]).norm() / full["ddt"].norm()).item()
    assert rel <= 1e-5  # two-part operands: 2^-16 of the terms, no rounding to bf16


@pytest.mark.gpu
def test_sequences_of_a_pack_alone():
    """A sequence's chunks are the same alone and in a pack, so its outputs are the same bits as
    long as its segments are (the pack's sequences here have one)."""
    a, grads, cu, softplus, _ = make("packed", 3)
    d, (y, ht) = forward(a, cu, softplus)
    got = backward(d, grads, cu, softplus)
    for n, (p, q) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        if p == q:
            assert torch.equal(ht[n], d["h0"][n]) and torch.equal(got["dh0"][n].cpu(), grads["dht"][n])
            continue
        one = {k: v[:, p:q].contiguous() if k in ("x", "dt", "B", "C") else v for k, v in d.items()}
        one["h0"] = d["h0"][n:n + 1]
        y1, h1 = kda.chunk_ssm(one["x"], one["dt"], one["A_log"], one["B"], one["C"], one["D"], one["dt_bias"], softplus, one["h0"], True)
        if q - p <= 256:
            assert torch.equal(y1, y[:, p:q]) and torch.equal(h1, ht[n:n + 1])
        near("y", y1, y[:, p:q].double().cpu(), torch.bfloat16)


@pytest.mark.gpu
def test_other_sequences_stay_clean():
    """A NaN and an infinity in one sequence (and in its state) reach no other."""
    a, grads, cu, softplus, _ = make("packed", 4)
    _, (y, ht) = forward(a, cu, softplus)
    clean = backward({k: on_gpu(v) for k, v in a.items()}, grads, cu, softplus)
    bad = {k: None if v is None else v.clone() for k, v in a.items()}
    bad["x"][0, 70, 1, 3], bad["B"][0, 100, 0, 5], bad["h0"][3] = float("nan"), float("inf"), float("nan")
    d, (y2, ht2) = forward(bad, cu, softplus)
    got = backward(d, grads, cu, softplus)
    keep = torch.ones(420, dtype=torch.bool)
    keep[64:129] = False
    others = [0, 1, 2, 4, 5, 6]
    assert torch.equal(y[:, keep], y2[:, keep]) and torch.equal(ht[others], ht2[others])
    for k in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(clean[k][:, keep], got[k][:, keep]), k
    assert torch.equal(clean["dh0"][others], got["dh0"][others])


@pytest.mark.gpu
def test_extreme_decays():
    """Steps from nothing to beyond every decay: what is forgotten is forgotten, what is not stays."""
    a, grads, _, _, t = make("a chunk and one", 5)
    a["dt"], a["dt_bias"] = torch.full_like(a["dt"], 0.01), None
    a["dt"][0, 20], a["dt"][0, 40], a["dt"][0, 41], a["dt"][0, 50] = 1000.0, 0.0, 3e4, 1e-30
    d, (y, ht) = forward(a, None, False)
    want, last = lo.ssm(a["x"], a["dt"], a["A_log"], a["B"], a["C"], a["D"], None, False, a["h0"])
    near("y", y, want, t)
    near("state", ht, last, t, True)
    got = backward(d, grads, None, False)
    full = lo.ssm_bwd(a["x"], a["dt"], a["A_log"], a["B"], a["C"], grads["dy"], grads["dht"], a["D"], None, False, a["h0"])
    for k in ("dx", "dB", "dC"):
        near(k, got[k], full[k], t)
    assert all(v.isfinite().all() for v in got.values())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,H,G,N,P,extra", [(1, 1, 1, 32, 32, 0), (9, 4, 2, 96, 64, 7), (5, 3, 1, 128, 96, 0), (200, 4, 4, 64, 128, 16)])
def test_step(kind, rows, H, G, N, P, extra):
    t, g = TYPES[kind], torch.Generator().manual_seed(6)
    pool = rows + 3
    a = dict(x=torch.randn(rows, 1, H, P, generator=g).to(t), dt=torch.randn(rows, 1, H, generator=g).to(t),
             B=torch.randn(rows, 1, G, N, generator=g).to(t), C=torch.randn(rows, 1, G, N, generator=g).to(t))
    A_log, D, bias = torch.rand(H, generator=g) * 2, torch.randn(H, generator=g), torch.randn(H, generator=g) - 2
    state = torch.randn(pool, H, N, P, generator=g)
    slots = torch.randperm(pool, generator=g)[:rows].to(torch.int32)
    if rows > 1:
        slots[0], slots[-1] = -1, pool
    d = {k: on_gpu(strided(v, extra, g))[:, 0] for k, v in a.items()}
    dev_state = state.to(DEV)
    y = kda.ssm_step(d["x"], d["dt"], A_log.to(DEV), d["B"], d["C"], dev_state, D.to(DEV), bias.to(DEV), True, slots.to(DEV))
    live = [(r, s) for r, s in enumerate(slots.tolist()) if 0 <= s < pool]
    at, of = [r for r, _ in live], [s for _, s in live]
    h = torch.finfo(t).eps / 2 if t == torch.bfloat16 else U
    args = ({k: v[at] for k, v in a.items()}, state[of])
    want, last = lo.ssm(args[0]["x"], args[0]["dt"], A_log, args[0]["B"], args[0]["C"], D, bias, True, args[1])
    size, size_last = lo.ssm(args[0]["x"].abs(), args[0]["dt"], A_log, args[0]["B"].abs(), args[0]["C"].abs(), D.abs(), bias, True, args[1].abs())
    c = (N + 60) * U  # the sum over N, and the decay's and step's own roundings
    check("y", y[at], want[:, 0], h * want[:, 0].abs() + c * size[:, 0])
    check("state", dev_state[of], last, 60 * U * size_last)
    others = [s for s in range(pool) if s not in of]
    assert torch.equal(dev_state[others].cpu(), state[others])
    assert all((y[r] == 0).all() for r in range(rows) if r not in at)


@pytest.mark.gpu
def test_steps_continue_a_prompt():
    a, _, _, softplus, t = make("a chunk and one", 7)
    d, (y, last) = forward(a, None, softplus)
    _, state = kda.chunk_ssm(d["x"][:, :50].contiguous(), d["dt"][:, :50].contiguous(), d["A_log"], d["B"][:, :50].contiguous(),
                             d["C"][:, :50].contiguous(), d["D"], d["dt_bias"], softplus, d["h0"], True)
    steps = [kda.ssm_step(d["x"][:, i], d["dt"][:, i], d["A_log"], d["B"][:, i], d["C"][:, i], state, d["D"], d["dt_bias"], softplus)
             for i in range(50, 65)]
    near("y", torch.stack(steps, 1), y[:, 50:].double().cpu(), t)
    near("state", state, last.double().cpu(), t, True)


@pytest.mark.gpu
@pytest.mark.parametrize("case", ["packed", "a chunk and one"])
def test_captured_and_replayed(case):
    a, grads, cu, softplus, _ = make(case, 8)
    d = {k: on_gpu(v) for k, v in a.items()}
    dy, dht, state = grads["dy"].to(DEV), grads["dht"].to(DEV), d["h0"].clone()
    cu_dev = None if cu is None else cu.to(DEV)

    def everything():
        y, ht = kda.chunk_ssm(d["x"], d["dt"], d["A_log"], d["B"], d["C"], d["D"], d["dt_bias"], softplus, d["h0"], True, cu_dev,
                              cu_seqlens_host=cu)
        g = kda.chunk_ssm_bwd(d["x"], d["dt"], d["A_log"], d["B"], d["C"], dy, dht, d["D"], d["dt_bias"], softplus, d["h0"], cu_dev,
                              cu_seqlens_host=cu)
        n = len(state)
        s = kda.ssm_step(d["x"][0, :n], d["dt"][0, :n], d["A_log"], d["B"][0, :n], d["C"][0, :n], state, d["D"], d["dt_bias"], softplus)
        return [y, ht, s, *g.values()]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything()
    side = torch.cuda.Stream()
    for seed in range(3):
        d["x"].copy_(torch.randn(d["x"].shape, generator=torch.Generator().manual_seed(seed)))
        state.copy_(d["h0"])
        graph.replay()
        torch.cuda.synchronize()
        got, moved = [v.clone() for v in out], state.clone()
        state.copy_(d["h0"])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = everything()
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(moved, state)


@pytest.mark.gpu
def test_refusals_on_the_device():
    z = dict(dtype=torch.float32, device=DEV)
    x, dt, A, B = torch.zeros(2, 6, 4, 32, **z), torch.zeros(2, 6, 4, **z), torch.zeros(4, **z), torch.zeros(2, 6, 2, 32, **z)
    st = torch.zeros(2, 4, 32, 32, **z)
    bad = [
        lambda: kda.chunk_ssm(x[..., :16].contiguous(), dt, A, B, B), lambda: kda.chunk_ssm(x, dt, A, B[..., :24].contiguous(), B[..., :24].contiguous()),
        lambda: kda.chunk_ssm(x, dt, A, torch.zeros(2, 6, 3, 32, **z), torch.zeros(2, 6, 3, 32, **z)),
        lambda: kda.chunk_ssm(x, dt, A, B, B[:, :5]), lambda: kda.chunk_ssm(x, dt, A, B, B.bfloat16()), lambda: kda.chunk_ssm(x, dt[..., :3], A, B, B),
        lambda: kda.chunk_ssm(x, dt, None, B, B), lambda: kda.chunk_ssm(x, dt, A.bfloat16(), B, B), lambda: kda.chunk_ssm(x, dt, A, B, B, D=A[:2]),
        lambda: kda.chunk_ssm(x.half(), dt, A, B.half(), B.half()), lambda: kda.chunk_ssm(x.transpose(2, 3), dt, A, B, B),
        lambda: kda.chunk_ssm(x, dt, A, B, B, initial_state=st[:1]), lambda: kda.chunk_ssm(x, dt, A, B, B, initial_state=st.bfloat16()),
        lambda: kda.chunk_ssm(x, dt, A, B, B, cu_seqlens=torch.tensor([0, 12])), lambda: kda.chunk_ssm(x[:0], dt[:0], A, B[:0], B[:0]),
        lambda: kda.chunk_ssm(torch.zeros(1, 1, 1, 160, **z), dt[:1, :1, :1], A[:1], B[:1, :1, :1], B[:1, :1, :1]),
        lambda: kda.chunk_ssm_bwd(x, dt, A, B, B, x.bfloat16()), lambda: kda.chunk_ssm_bwd(x, dt, A, B, B, x, dht=st[:, :2]),
        lambda: kda.ssm_step(x[:, 0], dt[:, 0], A, B[:, 0], B[:, 0], st[:1]), lambda: kda.ssm_step(x[:, 0], dt[:, 0], A, B[:, 0], B[:, 0], st.half()),
        lambda: kda.ssm_step(x[:, 0], dt[:, 0], A, B[:, 0], B[:, 0], st, slots=torch.zeros(2, dtype=torch.int64, device=DEV)),
    ]
    for f in bad:
        with pytest.raises(kda.KDAContractError):
            f()
