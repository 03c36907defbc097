"""The operators together, as a hybrid layer runs them on the GPU: RMS norm with the residual's
addition, a projection, the short convolution, the delta rule and the state space scan side by side on
slices of it, a gated sum and an RMS norm to 8 bits; prompts first, then single tokens out of state
pools, and the gradients through the chain.

Serving: every operator against its float64 definition on the inputs it really got, over the
whole stream of prompt and single tokens, so that a state left wrong by one call shows in the
next.  Bounds in the norm: a value's roundings are off by at most h = 2^-8 (bf16) of it each, the
three of an operand, a product and a store by h in the norm together (their root mean squares are
h / sqrt 3); fp32 chains of c <= 600 additions by sqrt c 2^-24 <= 1.5e-6.  The delta rule has the
bounds that its own tests hold it to: 1e-3 of the largest value in fp32, 2e-2 in the norm in bf16.
8-bit values are off by at most half a step, 2^-4, of themselves, or half of the smallest one, 2^-10
of their scale, besides the norm's h.

Training, in fp32: a stage adds at most 1.5e-6 in the norm and at most doubles what came before it
(it is a product with a matrix of near-orthogonal rows, a normalisation, a decaying sum), the delta rule
1e-4 (what its forms agree to in its own tests).  Behind the delta rule are the convolution, the projection and the
norm: 1e-4 * 2^3 + 1.5e-6 * 2^6 < 1e-3.  Differences of the float64 chain at +-e have an error of
e^2 / 6 of the third derivative, and 2^-52 / e of rounding: 1e-5 of the gradient for e = 1e-4.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gated_delta_rule_log2_amd as kda
from oracle import kda_oracle, kda_oracle_bwd, layer_oracle as lo

DEV = "cuda"
H, K, G = 2, 64, 1  # heads of either kind, their width (keys, values, state and channels), groups of B and C
DM, W = 128, 4      # the model's width, the convolution's
QKV, CONV = 3 * H * K, 3 * H * K + H * K + 2 * G * K
GATES = H * K + H + H  # g, beta, dt
EPS = 1e-5


def weights(t, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g) * std).to(dtype)

    return dict(norm=1 + normal(DM, std=0.1), proj=normal(DM, CONV + GATES, std=DM ** -0.5),
                conv=normal(CONV, W, std=W ** -0.5), conv_bias=normal(CONV, std=0.1), A_kda=torch.rand(H, generator=g),
                bias_kda=normal(H * K, std=0.5, dtype=torch.float32), A_ssm=torch.rand(H, generator=g) * 2,
                bias_ssm=normal(H, dtype=torch.float32) - 2, skip=normal(H, dtype=torch.float32), norm_out=1 + normal(H * K, std=0.1))


def slices(c, z):
    """q, k, v, x, B, C of the convolution's output and g, beta, dt of the projection's, as views."""
    lead = c.shape[:-1]
    q, k, v, x, B, C = c.split([H * K, H * K, H * K, H * K, G * K, G * K], -1)
    g, beta, dt = z[..., CONV:].split([H * K, H, H], -1)
    heads = [a.reshape(*lead, H, K).contiguous() for a in (q, k, v)]
    return heads, x.unflatten(-1, (H, K)), B.unflatten(-1, (G, K)), C.unflatten(-1, (G, K)), g.reshape(*lead, H, K).contiguous(), beta, dt


KDA_FLAGS = dict(use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True, use_beta_sigmoid_in_kernel=True)
KDA_ORACLE = dict(scale=K ** -0.5, gate_mode=kda_oracle.GATE_SOFTPLUS, qk_l2norm=True, beta_mode=kda_oracle.BETA_SIGMOID)


def project(n, w):
    return (n.reshape(-1, DM) @ w["proj"]).reshape(*n.shape[:-1], -1)


def prompt(x, residual, w, cu):
    n, h = kda.rms_norm(x, w["norm"], residual, EPS)
    z = project(n, w)
    dev_cu = cu.to(DEV)
    c, conv_state = kda.short_conv(z[..., :CONV], w["conv"], w["conv_bias"], "silu", None, True, dev_cu, cu_seqlens_host=cu)
    (q, k, v), xs, B, C, g, beta, dt = slices(c, z)
    o, kda_state = kda.chunk_kda(q, k, v, g, beta.contiguous(), output_final_state=True, cu_seqlens=dev_cu, A_log=w["A_kda"],
                                 dt_bias=w["bias_kda"], **KDA_FLAGS)
    y, ssm_state = kda.chunk_ssm(xs, dt, w["A_ssm"], B, C, w["skip"], w["bias_ssm"], True, None, True, dev_cu, cu_seqlens_host=cu)
    s = (o + y).flatten(2)
    return dict(h=h, n=n, z=z, c=c, o=o, y=y, s=s, out=kda.rms_norm_fp8(s, w["norm_out"], None, EPS, 64)), (conv_state, kda_state, ssm_state)


def token(x, residual, w, pools, slots, live):
    """One token of each row; rows at which `live` is false are padding."""
    conv_pool, kda_pool, ssm_pool = pools
    n, h = kda.rms_norm(x, w["norm"], residual, EPS)
    z = project(n, w)
    c = kda.short_conv_step(z[..., :CONV], conv_pool, w["conv"], w["conv_bias"], "silu", slots)
    (q, k, v), xs, B, C, g, beta, dt = slices(c, z)
    at = slots.long().clamp(min=0)
    o, ht = kda.fused_recurrent_kda(*(a.unsqueeze(1).contiguous() for a in (q, k, v, g, beta)), initial_state=kda_pool[at],
                                    output_final_state=True, A_log=w["A_kda"], dt_bias=w["bias_kda"], **KDA_FLAGS)
    kda_pool[at[live]] = ht[live]
    y = kda.ssm_step(xs, dt, w["A_ssm"], B, C, ssm_pool, w["skip"], w["bias_ssm"], True, slots)
    s = (o[:, 0] + y).flatten(1)
    return dict(h=h, n=n, z=z, c=c, o=o[:, 0], y=y, s=s, out=kda.rms_norm_fp8(s, w["norm_out"], None, EPS, 64))


def near(name, got, want, bound):
    got, want = got.double().cpu(), torch.as_tensor(np.asarray(want))
    rel = ((got - want).norm() / want.norm().clamp(min=1e-30)).item()
    assert got.shape == want.shape and rel <= bound, f"{name}: {rel:.3g} in the norm, bound {bound:.3g}"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_prompts_and_single_tokens(kind):
    t = torch.bfloat16 if kind == "bf16" else torch.float32
    bound = 2.0 ** -8 + 1.5e-6 if kind == "bf16" else 1.5e-6
    lengths, more = [5, 70, 0, 1, 200], 4
    cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int64)
    w = weights(t)
    wd = {k: v.to(DEV) for k, v in w.items()}
    g = torch.Generator().manual_seed(1)
    rows = len(lengths)
    xs = [torch.randn(2, n + more, DM, generator=g).to(t) for n in lengths]  # x and the residual of each sequence
    packed = torch.cat([a[:, :n] for a, n in zip(xs, lengths)], 1).to(DEV)
    first, states = prompt(packed[:1], packed[1:], wd, cu)

    # pools with more slots than rows, in another order; a padding row at the end
    order = torch.tensor([6, 2, 0, 5, 3])
    slots = torch.cat([order, torch.tensor([-1])]).to(torch.int32).to(DEV)
    pools = [torch.full((8, *s.shape[1:]), 7.0, dtype=s.dtype, device=DEV) for s in states]
    for pool, s in zip(pools, states):
        pool[order.to(DEV)] = s
    live = torch.arange(rows + 1, device=DEV) < rows
    steps = []
    for i in range(more):
        now = torch.stack([a[:, n + i] for a, n in zip(xs, lengths)] + [torch.zeros(2, DM, dtype=t)], 1).to(DEV)
        steps.append(token(now[0], now[1], wd, pools, slots, live))

    def stream(name, n):
        """What the operators put out for sequence n, over prompt and single tokens."""
        a, b = int(cu[n]), int(cu[n + 1])
        return torch.cat([first[name][:, a:b]] + [s[name][n][None, None] for s in steps], 1).cpu()

    for n in range(rows):
        z, c = stream("z", n), stream("c", n)
        h = xs[n][0] + xs[n][1]
        assert torch.equal(stream("h", n)[0], h)
        near("norm", stream("n", n)[0], lo.rms_norm(h, w["norm"], EPS), bound)
        want, last, _, _ = lo.short_conv(z[..., :CONV], w["conv"], w["conv_bias"], True)
        near("convolution", c, want, bound)
        assert torch.equal(pools[0][order[n]].cpu().double(), last[0])
        (q, k, v), x, B, C, gate, beta, dt = slices(c, z)
        want, last = kda_oracle.oracle_fwd(*(a.float().numpy() for a in (q, k, v, gate, beta)), A_log=w["A_kda"].numpy(),
                                           dt_bias=w["bias_kda"].numpy(), **KDA_ORACLE)
        size = np.abs(want).max()
        if kind == "fp32":
            assert np.abs(stream("o", n).numpy() - want).max() <= 1e-3 * max(size, 1) and np.abs(pools[1][order[n]].cpu().numpy() - last[0]).max() <= 1e-3
        else:
            near("delta rule", stream("o", n), want, 2e-2)
            near("its state", pools[1][order[n]], last[0], 2e-2)
        want, last = lo.ssm(x, dt, w["A_ssm"], B, C, w["skip"], w["bias_ssm"], True)
        near("scan", stream("y", n), want, bound)
        near("its state", pools[2][order[n]], last[0], 1.5e-6)
        a, b = int(cu[n]), int(cu[n + 1])
        q8 = torch.cat([first["out"][0][0, a:b].float()] + [s["out"][0][n][None].float() for s in steps]).cpu().double()
        scale = torch.cat([first["out"][1][0, a:b]] + [s["out"][1][n][None] for s in steps]).cpu().double().repeat_interleave(64, 1)
        want = lo.rms_norm(stream("s", n)[0], w["norm_out"], EPS)
        off = (q8 * scale - want).abs() - (2.0 ** -4 + 2.0 ** -20) * want.abs() - 2.0 ** -10 * scale
        assert off.max() <= 0
    # padding wrote nothing: its row is 0 where an operator says so, and unused slots are as they were
    assert not steps[-1]["c"][-1].any() and not steps[-1]["y"][-1].any()
    for pool in (pools[0], pools[2]):
        assert (pool[[1, 4, 7]] == 7).all()


def chain64(p, x, residual, u, starts):
    """<u, out> of the layer (without the 8 bits), differentiable, in float64."""
    h = x + residual
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * p["norm"]
    z = n @ p["proj"]
    outs = []
    for a, b in zip(starts, starts[1:]):
        zc = torch.cat([torch.zeros(W - 1, CONV, dtype=torch.float64), z[a:b, :CONV]])
        pre = p["conv_bias"] + sum(p["conv"][:, k] * zc[k:k + b - a] for k in range(W))
        c = pre * torch.sigmoid(pre)
        (q, k, v), xs, B, C, g, beta, dt = slices(c, z[a:b])
        o, _ = kda_oracle_bwd.forward(q, k, v, g, beta, A_log=p["A_kda"], dt_bias=p["bias_kda"], seq_starts=[0, b - a],
                                      scale=K ** -0.5, gate_mode=kda_oracle_bwd.GATE_SOFTPLUS, qk_l2norm=True,
                                      beta_mode=kda_oracle_bwd.BETA_SIGMOID)
        d = torch.nn.functional.softplus(dt + p["bias_ssm"], threshold=1e9)
        S = torch.zeros(H, K, K, dtype=torch.float64)
        y = []
        for i in range(b - a):
            S = torch.exp(-torch.exp(p["A_ssm"]) * d[i])[:, None, None] * S + d[i][:, None, None] * B[i, :, :, None] * xs[i][:, None, :]
            y.append((S * C[i, :, :, None]).sum(1) + p["skip"][:, None] * xs[i])
        s = (o + torch.stack(y)).flatten(1)
        outs.append(s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * p["norm_out"])
    return (torch.cat(outs) * u).sum()


def gradients(x, residual, w, u, cu):
    """The same chain and its gradients by the package's entries, from the last operator to the first."""
    dev_cu = cu.to(DEV)
    n, h = kda.rms_norm(x, w["norm"], residual, EPS)
    z = project(n, w)
    c, _ = kda.short_conv(z[..., :CONV], w["conv"], w["conv_bias"], "silu", cu_seqlens=dev_cu, cu_seqlens_host=cu)
    (q, k, v), xs, B, C, g, beta, dt = slices(c, z)
    beta = beta.contiguous()
    o, _ = kda.chunk_kda(q, k, v, g, beta, cu_seqlens=dev_cu, A_log=w["A_kda"], dt_bias=w["bias_kda"], **KDA_FLAGS)
    y, _ = kda.chunk_ssm(xs, dt, w["A_ssm"], B, C, w["skip"], w["bias_ssm"], True, None, False, dev_cu, cu_seqlens_host=cu)
    s = (o + y).flatten(2)
    _, s = kda.rms_norm(s, w["norm_out"], None, EPS)

    last = kda.rms_norm_bwd(s, w["norm_out"], u, None, EPS)
    ds = last["dx"].unflatten(-1, (H, K))
    a = kda.chunk_kda_bwd(q, k, v, g, beta, ds, cu_seqlens=dev_cu, A_log=w["A_kda"], dt_bias=w["bias_kda"], **KDA_FLAGS)
    b = kda.chunk_ssm_bwd(xs, dt, w["A_ssm"], B, C, ds, None, w["skip"], w["bias_ssm"], True, None, dev_cu, cu_seqlens_host=cu)
    dc = torch.cat([t.flatten(2).float() for t in (a["dq"], a["dk"], a["dv"], b["dx"], b["dB"], b["dC"])], -1)
    conv = kda.short_conv_bwd(z[..., :CONV], w["conv"], dc, w["conv_bias"], "silu", cu_seqlens=dev_cu, cu_seqlens_host=cu)
    dz = torch.cat([t.to(x.dtype) for t in (conv["dx"], a["dg"].flatten(2), a["dbeta"], b["ddt"])], -1)
    dn = (dz.flatten(0, 1) @ w["proj"].t().contiguous()).reshape(n.shape)
    first = kda.rms_norm_bwd(h, w["norm"], dn, None, EPS)
    grads = dict(x=first["dx"][0], norm=first["dweight"], proj=n.flatten(0, 1).t().contiguous() @ dz.flatten(0, 1),
                 conv=conv["dweight"], conv_bias=conv["dbias"], A_kda=a["dA_log"], bias_kda=a["ddt_bias"], A_ssm=b["dA_log"],
                 bias_ssm=b["ddt_bias"], skip=b["dD"], norm_out=last["dweight"])
    return grads, z, dc, conv


@pytest.mark.gpu
def test_gradients_through_the_chain():
    lengths = [40, 1, 90]
    cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int64)
    w = weights(torch.float32, 2)
    g = torch.Generator().manual_seed(3)
    x, residual, u = torch.randn(3, 1, sum(lengths), DM, generator=g)
    got, *_ = gradients(x.to(DEV), residual.to(DEV), {k: v.to(DEV) for k, v in w.items()}, u.to(DEV), cu)
    p = {k: v.double().requires_grad_() for k, v in w.items()}
    x64 = x[0].double().requires_grad_()
    starts = cu.tolist()
    chain64(p, x64, residual[0].double(), u[0].double(), starts).backward()
    want = dict({k: v.grad for k, v in p.items()}, x=x64.grad)
    assert set(got) == set(want)
    for k in want:
        near(k, got[k].reshape(want[k].shape), want[k], 1e-3)
    # along a direction of every input at once, against differences
    e, direction = 1e-4, {k: torch.randn(v.shape, generator=g).double() * (v.detach().abs().mean() + 0.1) for k, v in dict(p, x=x64).items()}
    with torch.no_grad():
        at = [chain64({k: v + f * e * direction[k] for k, v in p.items()}, x64 + f * e * direction["x"], residual[0].double(),
                      u[0].double(), starts) for f in (1, -1)]
    slope = (at[0] - at[1]).item() / (2 * e)
    parts = {k: (got[k].reshape(want[k].shape).double().cpu() * direction[k]).sum().item() for k in want}
    size = sum(want[k].norm().item() * direction[k].norm().item() for k in want)
    assert abs(sum(parts.values()) - slope) <= 1e-3 * size + 1e-5 * abs(slope)


@pytest.mark.gpu
def test_the_delta_rules_gradients_reach_a_convolution_in_16_bits():
    """The delta rule's gradients leave in 32 bits and enter the convolution's backward so: off by the roundings
    of dx at its store, h of it, the weights' sums by sqrt(tokens) 2^-24 only."""
    lengths = [33, 0, 100]
    cu = torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int64)
    w = weights(torch.bfloat16, 4)
    g = torch.Generator().manual_seed(5)
    x, residual, u = torch.randn(3, 1, sum(lengths), DM, generator=g).to(torch.bfloat16).to(DEV)
    _, z, dc, conv = gradients(x, residual, {k: v.to(DEV) for k, v in w.items()}, u, cu)
    assert dc.dtype == torch.float32
    want, _ = lo.short_conv_bwd(z[..., :CONV], w["conv"], dc, w["conv_bias"], True, cu=cu)
    near("dx", conv["dx"], want["dx"], 2.0 ** -8)
    near("dweight", conv["dweight"], want["dweight"], 1.5e-6)
    near("dbias", conv["dbias"], want["dbias"], 1.5e-6)
