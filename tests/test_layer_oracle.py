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
