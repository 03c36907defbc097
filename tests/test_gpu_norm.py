"""The RMS norm on the GPU against its float64 definition (oracle/layer_oracle.py).

Tolerances count roundings, u = 2^-24 for one in fp32 and half a step of the output's type for
the store.  The sum of D squares is off by at most n u of itself, n the longest chain of
additions: 32 in a thread, 6 across lanes, 16 across waves.  Its square root halves that, and
the division by D, eps, the root, the reciprocal and the two products add 6 u.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_log2_amd as kda
from oracle import layer_oracle as lo

DEV = "cuda"
U = 2.0 ** -24
CHAIN = 32 + 6 + 16
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZES = [(1, 1), (3, 7), (5, 8), (1, 64), (130, 100), (6, 512), (9, 513), (3, 1024), (7, 1500), (5, 2048), (17, 4096),
         (3, 4099), (2, 8192), (2, 8200), (2, 20000), (1, 32768), (2100, 640)]


def make(rows, D, kind, seed=0, wide_weight=True):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[kind]
    w = torch.rand(D, generator=g) + 0.5
    return dict(x=torch.randn(rows, D, generator=g).to(t), residual=(3 * torch.randn(rows, D, generator=g)).to(t),
                weight=w if wide_weight else w.to(torch.bfloat16), dy=torch.randn(rows, D, generator=g).to(t),
                dh=torch.randn(rows, D, generator=g).to(t))


def check(name, got, want, bound):
    off = (got.double().cpu() - want).abs()
    worst = (off / bound.clamp(min=1e-300)).max().item()
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,D", SIZES)
def test_forward(rows, D, kind):
    a = make(rows, D, kind, wide_weight=D % 2 == 0)
    d = {k: v.to(DEV) for k, v in a.items()}
    t = TYPES[kind]
    y, same = kda.rms_norm(d["x"], d["weight"], eps=1e-5)
    assert same is d["x"]
    want = lo.rms_norm(a["x"], a["weight"], 1e-5)
    check("y", y, want, (torch.finfo(t).eps / 2 + (CHAIN / 2 + 6) * U) * want.abs() + 1e-30)
    y, h = kda.rms_norm(d["x"], d["weight"], d["residual"], eps=1e-5)
    sums = (a["x"].float() + a["residual"].float()).to(t)  # one rounding in fp32, one in the type
    assert torch.equal(h.cpu(), sums)
    want = lo.rms_norm(sums, a["weight"], 1e-5)
    check("y", y, want, (torch.finfo(t).eps / 2 + (CHAIN / 2 + 6) * U) * want.abs() + 1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,D,group", [(1, 64, 0), (3, 7, 0), (5, 100, 0), (5, 4099, 0), (2, 20000, 0), (9, 512, 512),
                                          (33, 4096, 128), (7, 640, 32), (4, 1536, 512), (3, 8192, 64), (2, 32768, 128),
                                          (6, 72, 8), (4, 48, 16)])
def test_eight_bits(rows, D, group, kind):
    """Scales to fp32 roundings; every code within half a step of the value that it stands for.
    (y / scale is off by (CHAIN / 2 + 10) u of itself before its rounding, which can only move
    a value that close to the middle between two codes to the other of them.)"""
    a = make(rows, D, kind, 1)
    a["x"][0, :min(D, group or D)] = 0
    a["residual"][0, :min(D, group or D)] = 0  # a group of zeros
    q, scales, h = kda.rms_norm_fp8(a["x"].to(DEV), a["weight"].to(DEV), a["residual"].to(DEV), 1e-5, group)
    sums = (a["x"].float() + a["residual"].float()).to(TYPES[kind])
    assert torch.equal(h.cpu(), sums)
    want = lo.rms_norm(sums, a["weight"], 1e-5).reshape(rows, -1, group or D)
    big = want.abs().amax(2).clamp(min=1e-30)
    off = (CHAIN / 2 + 10) * U
    check("scales", scales, big / 448, off * big / 448)
    value = want / (big / 448)[..., None]
    codes = lo.e4m3_values()
    at = torch.searchsorted(codes, value.contiguous()).clamp(1, len(codes) - 1)
    low, high = codes[at - 1], codes[at]
    got = q.double().cpu().reshape(value.shape)
    assert ((got == low) | (got == high) | (value.abs() >= 448)).all()
    assert ((got - value).abs() <= (high - low) / 2 + off * value.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,D", SIZES)
def test_backward(rows, D, kind):
    """dx carries the errors of both sums: of g h (CHAIN + 3 roundings of its terms' sizes) and
    of h^2 in r^3 (three halves of CHAIN); dweight a chain over the rows of a workgroup and the
    partials of at most 1024 of them, its terms off by r's error and 3 u."""
    a = make(rows, D, kind, 2, wide_weight=D % 2 == 0)
    d = {k: v.to(DEV) for k, v in a.items()}
    t = TYPES[kind]
    for dh in (None, "dh"):
        got = kda.rms_norm_bwd(d["x"], d["weight"], d["dy"], None if dh is None else d["dh"], 1e-5)
        want, sizes = lo.rms_norm_bwd(a["x"], a["weight"], a["dy"], 1e-5, None if dh is None else a["dh"])
        check("dx", got["dx"], want["dx"], torch.finfo(t).eps / 2 * want["dx"].abs() + (2.5 * CHAIN + 20) * U * sizes["dx"] + 1e-30)
        chain = min(rows, 1024) + rows / 256 + CHAIN / 2 + 12
        check("dweight", got["dweight"], want["dweight"], chain * U * sizes["dweight"] + 1e-30)
        assert got["dx"].dtype == t and got["dweight"].dtype == torch.float32


@pytest.mark.gpu
def test_no_rows_and_leading_dimensions():
    w = torch.rand(96, device=DEV)
    y, h = kda.rms_norm(torch.empty(0, 96, device=DEV), w, torch.empty(0, 96, device=DEV))
    assert y.shape == h.shape == (0, 96)
    g = kda.rms_norm_bwd(torch.empty(0, 96, device=DEV), w, torch.empty(0, 96, device=DEV))
    assert (g["dweight"] == 0).all()
    x = torch.randn(2, 3, 5, 96, device=DEV)
    y, _ = kda.rms_norm(x, w)
    assert torch.equal(y.reshape(30, 96), kda.rms_norm(x.reshape(30, 96), w)[0])
    q, s, _ = kda.rms_norm_fp8(x, w, group_size=32)
    assert q.shape == x.shape and s.shape == (2, 3, 5, 3)


@pytest.mark.gpu
def test_zeros_nan_and_infinities():
    x = torch.ones(4, 256, device=DEV)
    x[1], x[2, 7], x[3, 9] = 0, float("nan"), float("inf")
    w = torch.ones(256, device=DEV)
    y, _ = kda.rms_norm(x, w, eps=0.0)
    assert (y[0] == 1).all() and y[1].isnan().all() and y[2].isnan().all() and y[3, 9].isnan() and (y[3, :9] == 0).all()
    q, s, _ = kda.rms_norm_fp8(x, w, eps=1e-6, group_size=128)
    assert (q[1].float() == 0).all() and s[1].isfinite().all()
    assert s[2].isnan().all() and q[2].float().isnan().all()
    assert s[3, 0].isnan() and s[3, 1].isfinite()
    assert ((q[0].float() * s[0].repeat_interleave(128) - 1).abs() < 1e-6).all()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    a = {k: v.to(DEV) for k, v in make(70, 4096, "bf16", 3).items()}

    def everything():
        y, h = kda.rms_norm(a["x"], a["weight"], a["residual"])
        q, s, _ = kda.rms_norm_fp8(a["x"], a["weight"], a["residual"], group_size=128)
        return [y, h, q.view(torch.uint8), s, *kda.rms_norm_bwd(h, a["weight"], a["dy"], a["dh"]).values()]

    everything()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything()
    side = torch.cuda.Stream()
    for seed in range(3):
        a["x"].copy_(torch.randn(a["x"].shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        with torch.cuda.stream(side):
            want = everything()
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
def test_refusals_on_the_device():
    x, w = torch.zeros(4, 96, device=DEV), torch.zeros(96, device=DEV)
    for f in (lambda: kda.rms_norm(x.half(), w), lambda: kda.rms_norm(x, w[:95]), lambda: kda.rms_norm(x.t(), w[:4]),
              lambda: kda.rms_norm(x, w, x[:3]), lambda: kda.rms_norm(x, w, x.bfloat16()), lambda: kda.rms_norm(x, w, eps=-1.0),
              lambda: kda.rms_norm_fp8(x, w, group_size=64), lambda: kda.rms_norm_fp8(x, w, group_size=24),
              lambda: kda.rms_norm_fp8(x, w, group_size=-1), lambda: kda.rms_norm_bwd(x, w, x.bfloat16()),
              lambda: kda.rms_norm_bwd(x, w, x, x[:2]), lambda: kda.rms_norm(x, w.cpu()),
              lambda: kda.rms_norm(torch.zeros(1, 32776, device=DEV), torch.zeros(32776, device=DEV))):
        with pytest.raises(kda.KDAContractError):
            f()
