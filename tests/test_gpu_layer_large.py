"""The layer's operators where elements lie more than 2^31 from a tensor's first: the same values, bit for
bit, as on compact copies of the part that is compared.  Most of the memory is never touched.
"""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_log2_amd as kda

DEV = "cuda"
BF = torch.bfloat16


def normal(*shape, dtype=BF, std=1.0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def far_apart(v, stride):
    """v [1, T, ...] as a view whose tokens lie `stride` elements apart."""
    T = v.shape[1]
    base = torch.empty((T - 1) * stride + v[0, 0].numel(), dtype=v.dtype, device=DEV)
    strides = [(T - 1) * stride + v[0, 0].numel(), stride]
    inner = 1
    tail = []
    for n in reversed(v.shape[2:]):
        tail.insert(0, inner)
        inner *= n
    return base.as_strided(v.shape, strides + tail).copy_(v)


@pytest.mark.gpu
def test_convolution_over_long_strides():
    T, D, stride = 2100, 72, (1 << 20) + 8
    x, w, dy = normal(1, T, D), normal(D, 4), normal(1, T, D, seed=1)
    far = far_apart(x, stride)
    assert (T - 1) * stride > 1 << 31
    cu = torch.tensor([0, 1500, T])
    a, b = (kda.short_conv(t, w, None, "silu", None, True, cu.to(DEV), cu_seqlens_host=cu) for t in (x, far))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = (kda.short_conv_bwd(t, w, dy, None, "silu", cu_seqlens=cu.to(DEV), cu_seqlens_host=cu) for t in (x, far))
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
def test_convolution_of_many_values():
    T, D, tail = 270000, 8000, 1000
    assert T * D > 1 << 31
    x = torch.zeros(1, T, D, dtype=BF, device=DEV)
    dy = torch.zeros(1, T, D, dtype=BF, device=DEV)
    x[:, -tail:], dy[:, -tail:] = normal(1, tail, D), normal(1, tail, D, seed=1)
    w = normal(D, 4)
    y, last = kda.short_conv(x, w, None, "silu", None, True)
    ys, lasts = kda.short_conv(x[:, -tail:].contiguous(), w, None, "silu", None, True)
    assert torch.equal(y[:, -tail:], ys) and torch.equal(last, lasts) and not y[:, :-tail].any()
    del y
    dx = kda.short_conv_bwd(x, w, dy, None, "silu")["dx"]
    assert torch.equal(dx[:, -tail:], kda.short_conv_bwd(x[:, -tail:].contiguous(), w, dy[:, -tail:].contiguous(), None, "silu")["dx"])


@pytest.mark.gpu
def test_norm_of_many_values():
    rows, D, tail = 70000, 31000, 64
    assert rows * D > 1 << 31
    x = torch.empty(rows, D, dtype=BF, device=DEV)
    x[:-tail] = 1
    x[-tail:] = normal(tail, D)
    w = normal(D)
    y, _ = kda.rms_norm(x, w)
    assert torch.equal(y[-tail:], kda.rms_norm(x[-tail:].contiguous(), w)[0])
    q, scales, _ = kda.rms_norm_fp8(x, w, group_size=8)
    qs, scales_s, _ = kda.rms_norm_fp8(x[-tail:].contiguous(), w, group_size=8)
    assert torch.equal(q[-tail:].view(torch.uint8), qs.view(torch.uint8)) and torch.equal(scales[-tail:], scales_s)
    dx = kda.rms_norm_bwd(x, w, y)["dx"]
    assert torch.equal(dx[-tail:], kda.rms_norm_bwd(x[-tail:].contiguous(), w, y[-tail:].contiguous())["dx"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "fp32"])
def test_scan_over_the_longest_strides(dtype):
    """Strides of 2^24 - 1 elements: a chunk's offsets reach 2^30 elements, 2^31 bytes."""
    T, H, G, N, P, stride = 300, 2, 1, 32, 32, (1 << 24) - 1
    x, B, C = normal(1, T, H, P, dtype=dtype), normal(1, T, G, N, dtype=dtype, std=0.4, seed=1), normal(1, T, G, N, dtype=dtype, std=0.4, seed=2)
    dt, A, dy = normal(1, T, H, dtype=dtype, seed=3), torch.rand(H, device=DEV), normal(1, T, H, P, dtype=dtype, seed=4)
    dt_far = far_apart(dt, 1 << 23)
    want = kda.chunk_ssm(x, dt, A, B, C, None, None, True, None, True)
    grads = kda.chunk_ssm_bwd(x, dt, A, B, C, dy, None, None, None, True)
    for name in ("x", "B", "C"):
        t = dict(x=x, B=B, C=C)
        t[name] = far_apart(t[name], stride)
        assert (T - 1) * stride > 1 << 31
        got = kda.chunk_ssm(t["x"], dt_far, A, t["B"], t["C"], None, None, True, None, True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g = kda.chunk_ssm_bwd(t["x"], dt_far, A, t["B"], t["C"], dy, None, None, None, True)
        assert all(torch.equal(g[k], grads[k]) for k in grads)
        del t, got, g


@pytest.mark.gpu
def test_scan_of_many_values():
    """Nothing but zeros in front of the last tokens, which are then as alone, to the roundings: the chunks
    are divided differently there, states differ by fp32's, outputs by their store's (2^-8 of each)."""
    T, H, G, N, P, tail = 140032, 128, 8, 32, 128, 640
    assert T * H * P > 1 << 31 and (T - tail) % 64 == 0
    x, dy = (torch.zeros(1, T, H, P, dtype=BF, device=DEV) for _ in range(2))
    x[:, -tail:], dy[:, -tail:] = normal(1, tail, H, P), normal(1, tail, H, P, seed=1)
    B, C, dt = normal(1, T, G, N, std=0.4, seed=2), normal(1, T, G, N, std=0.4, seed=3), normal(1, T, H, seed=4)
    A, skip = torch.rand(H, device=DEV), torch.rand(H, device=DEV)
    end = [t[:, -tail:].contiguous() for t in (x, dt, B, C, dy)]
    y, last = kda.chunk_ssm(x, dt, A, B, C, skip, None, True, None, True)
    ys, lasts = kda.chunk_ssm(end[0], end[1], A, end[2], end[3], skip, None, True, None, True)
    assert not y[:, :-tail].any()
    near = lambda a, b, bound: (a.double() - b.double()).norm() <= bound * b.double().norm()  # noqa: E731
    assert near(y[:, -tail:], ys, 2.0 ** -8) and near(last, lasts, 1.5e-6)
    del y
    g = kda.chunk_ssm_bwd(x, dt, A, B, C, dy, None, skip, None, True)
    gs = kda.chunk_ssm_bwd(end[0], end[1], A, end[2], end[3], end[4], None, skip, None, True)
    for k in ("dx", "dB", "dC", "ddt"):
        assert near(g[k][:, -tail:], gs[k], 2.0 ** -8), k
    # the steps in front of them have no part: no state, no output
    assert not g["dC"][:, :-tail].any() and not g["ddt"][:, :-tail].any()


@pytest.mark.gpu
def test_steps_out_of_large_pools():
    rows, H, N, P = 5, 2, 128, 128
    slots = torch.tensor([0, 69999, 65535, 65536, 33333], dtype=torch.int32, device=DEV)
    pool = torch.empty(70000, H, N, P, device=DEV)
    assert pool.numel() > 1 << 31
    small = normal(rows, H, N, P, dtype=torch.float32)
    pool[slots.long()] = small
    x, dt, B, C, A = normal(rows, H, P), normal(rows, H, seed=1), normal(rows, 1, N, seed=2), normal(rows, 1, N, seed=3), torch.rand(H, device=DEV)
    y = kda.ssm_step(x, dt, A, B, C, pool, None, None, True, slots)
    assert torch.equal(y, kda.ssm_step(x, dt, A, B, C, small, None, None, True)) and torch.equal(pool[slots.long()], small)
    del pool
    D = 10240
    pool = torch.empty(70001, 3, D, dtype=BF, device=DEV)
    assert pool.numel() > 1 << 31
    small, x, w = normal(rows, 3, D), normal(rows, D, seed=1), normal(D, 4, seed=2)
    pool[slots.long()] = small
    y = kda.short_conv_step(x, pool, w, None, "silu", slots)
    assert torch.equal(y, kda.short_conv_step(x, small, w, None, "silu")) and torch.equal(pool[slots.long()], small)
