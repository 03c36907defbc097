"""The float64 definitions of the layer operators (oracle/layer_oracle.py) against values that
do not come from them: hand-worked sums, central differences, torch's own differentiation and
conversions."""
import pytest
import torch

from oracle import layer_oracle as lo


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_conv_by_hand():
    # one channel, weights (1, 10, 100) from the oldest input to the newest, state (7, 8)
    x = torch.tensor([[[1.0], [2.0], [3.0]]])
    y, last, _, _ = lo.short_conv(x, torch.tensor([[1.0, 10.0, 100.0]]), torch.tensor([0.5]), False,
                                  torch.tensor([[[7.0], [8.0]]]))
    assert y[0, :, 0].tolist() == [7 + 80 + 100 + 0.5, 8 + 10 + 200 + 0.5, 1 + 20 + 300 + 0.5]
    assert last[0, :, 0].tolist() == [2.0, 3.0]
    y, last, _, _ = lo.short_conv(x, torch.tensor([[1.0, 10.0, 100.0]]), cu=[0, 1, 1, 3])
    assert y[0, :, 0].tolist() == [100.0, 200.0, 320.0]
    assert last[:, :, 0].tolist() == [[0.0, 1.0], [0.0, 0.0], [2.0, 3.0]]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 6, 8]])
def test_conv_gradients_by_differences(silu, cu):
    B, T, D, W = (2, 5, 3, 4) if cu is None else (1, 8, 3, 4)
    n = B if cu is None else len(cu) - 1
    at = dict(x=rand(B, T, D, seed=1), weight=rand(D, W, seed=2), bias=rand(D, seed=3), h0=rand(n, W - 1, D, seed=4))
    dy, dht = rand(B, T, D, seed=5), rand(n, W - 1, D, seed=6)
    got, _ = lo.short_conv_bwd(at["x"], at["weight"], dy, at["bias"], silu, at["h0"], dht, cu)

    def loss(v):
        y, last, _, _ = lo.short_conv(v["x"], v["weight"], v["bias"], silu, v["h0"], cu)
        return (y * dy).sum() + (last * dht).sum()

    for k, name in dict(x="dx", weight="dweight", bias="dbias", h0="dh0").items():
        way, step = rand(*at[k].shape, seed=7), 1e-6
        up, down = dict(at, **{k: at[k] + step * way}), dict(at, **{k: at[k] - step * way})
        diff = (loss(up) - loss(down)) / (2 * step)
        assert abs(diff - (got[name] * way).sum()) <= 1e-7 * (1 + abs(diff)), name


def test_norm_gradients_by_torch():
    h, w, dy, dh = rand(6, 10, seed=1).requires_grad_(), rand(10, seed=2).requires_grad_(), rand(6, 10, seed=3), rand(6, 10, seed=4)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-3) * w
    assert torch.allclose(y, lo.rms_norm(h, w, 1e-3), rtol=0, atol=1e-14)
    dx, dw = torch.autograd.grad((y * dy).sum() + (h * dh).sum(), [h, w])
    got, _ = lo.rms_norm_bwd(h, w, dy, 1e-3, dh)
    assert torch.allclose(got["dx"], dx, rtol=0, atol=1e-13) and torch.allclose(got["dweight"], dw, rtol=0, atol=1e-13)


def test_e4m3_values_are_torch_codes():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[~codes.isnan()].unique()
    assert torch.equal(codes, lo.e4m3_values())


def test_ssm_by_hand():
    # one head, one state row, one channel; step 1 and A = -ln 2: S halves, then takes B x
    x, dt = torch.tensor([8.0, 4.0, 2.0]).view(1, 3, 1, 1), torch.ones(1, 3, 1)
    B, C = torch.tensor([1.0, 2.0, 3.0]).view(1, 3, 1, 1), torch.tensor([1.0, 1.0, 10.0]).view(1, 3, 1, 1)
    A_log = torch.log(torch.log(torch.tensor([2.0], dtype=torch.float64)))
    y, last = lo.ssm(x, dt, A_log, B, C, D=torch.tensor([0.5]), h0=torch.full((1, 1, 1, 1), 16.0))
    # S: 16/2 + 8 = 16; 8 + 8 = 16; 8 + 6 = 14
    assert torch.allclose(y.flatten(), torch.tensor([16 + 4.0, 16 + 2.0, 140 + 1.0], dtype=torch.float64), atol=1e-12, rtol=0)
    assert abs(last.item() - 14) < 1e-12
    y, last = lo.ssm(x, dt, A_log, B, C, cu=[0, 0, 1, 3])
    assert torch.allclose(y.flatten(), torch.tensor([8.0, 8.0, 100.0], dtype=torch.float64), atol=1e-12, rtol=0)
    assert torch.allclose(last.flatten(), torch.tensor([0.0, 8.0, 10.0], dtype=torch.float64), atol=1e-12, rtol=0)


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 9]])
def test_ssm_gradients_by_differences(softplus, cu):
    nb, T, H, G, N, P = (2, 6, 4, 2, 3, 5) if cu is None else (1, 9, 4, 2, 3, 5)
    n = nb if cu is None else len(cu) - 1
    at = dict(x=rand(nb, T, H, P, seed=1), dt=rand(nb, T, H, seed=2).abs() * 0.3, A_log=rand(H, seed=3) * 0.3,
              B=rand(nb, T, G, N, seed=4), C=rand(nb, T, G, N, seed=5), D=rand(H, seed=6), dt_bias=rand(H, seed=7) * 0.1,
              h0=rand(n, H, N, P, seed=8))
    dy, dht = rand(nb, T, H, P, seed=9), rand(n, H, N, P, seed=10)
    got = lo.ssm_bwd(at["x"], at["dt"], at["A_log"], at["B"], at["C"], dy, dht, at["D"], at["dt_bias"], softplus, at["h0"], cu)

    def loss(v):
        y, last = lo.ssm(v["x"], v["dt"], v["A_log"], v["B"], v["C"], v["D"], v["dt_bias"], softplus, v["h0"], cu)
        return (y * dy).sum() + (last * dht).sum()

    for k in at:
        way, step = rand(*at[k].shape, seed=11), 1e-6
        diff = (loss(dict(at, **{k: at[k] + step * way})) - loss(dict(at, **{k: at[k] - step * way}))) / (2 * step)
        mine = (got["d" + k] * way).sum()
        assert abs(diff - mine) <= 1e-6 * (1 + abs(diff)), (k, diff.item(), mine.item())
