"""The layer operators beside the delta attention, on real work: the short causal convolution, the selective
state space scan and the RMS norm with the residual's addition, each for prompts, for single tokens and for
their gradients.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, logarithms of decays in 64)
where `own` is false, and through this package's entry points where it is true.  `exact` has the values from the
definitions, token by token, in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64  # of the plain scan


def listed():
    return [
        # decoding: the convolution in front of q, k and v of the 16 / 32 head layer (2048 + 2048 + 4096 channels)
        # for 64 requests whose states lie in a pool of 256 slots
        dict(name="conv_step", op="conv_step", type="bf16", rows=64, slots=256, D=8192, W=4, silu=True),
        # a prompt pass over packed requests of different lengths: the value channels (32 heads of 128)
        dict(name="conv_packed", op="conv", type="bf16", B=1, T=8192, D=4096, W=4, silu=True, seqs=11, bias=False),
        # odd sizes without an activation, in 32 bits, two rows of a batch
        dict(name="conv_odd_f32", op="conv", type="fp32", B=2, T=1009, D=1000, W=3, silu=False, seqs=0, bias=True),
        # training: gradients of the same convolution
        dict(name="conv_bwd", op="conv_bwd", type="bf16", B=1, T=8192, D=4096, W=4, silu=True, seqs=0, bias=True),
        # a long prompt through the scan with the head layout of the grouped-value configuration
        dict(name="scan_gva", op="scan", type="bf16", B=1, T=8192, H=32, G=16, N=128, P=128, seqs=0),
        # packed requests that continue from their states, heads of 64 that share few B and C
        dict(name="scan_packed", op="scan", type="bf16", B=1, T=6000, H=64, G=8, N=128, P=64, seqs=13),
        # training: every gradient of the scan
        dict(name="scan_bwd_gva", op="scan_bwd", type="bf16", B=1, T=8192, H=32, G=16, N=128, P=128, seqs=0),
        # training in 32 bits, a batch of ragged length
        dict(name="scan_bwd_f32", op="scan_bwd", type="fp32", B=2, T=1003, H=8, G=2, N=64, P=64, seqs=0),
        # decoding: one token of 64 requests, states in a pool
        dict(name="scan_step", op="scan_step", type="bf16", rows=64, slots=96, H=32, G=16, N=128, P=128),
        # decoding: the pre-norm of 16 requests
        dict(name="norm_rows16", op="norm", type="bf16", rows=16, D=4096, quant=-1, residual=True),
        # a prompt's pre-norm whose output feeds an 8-bit projection, a scale for each 128 values
        dict(name="norm_fp8", op="norm", type="bf16", rows=8192, D=4096, quant=128, residual=True),
        # training: the norm's gradients, with the gradient that arrives at the residual
        dict(name="norm_bwd", op="norm_bwd", type="bf16", rows=8192, D=4096, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_bwd", "conv_step", "scan", "scan", "scan_bwd", "scan_bwd", "scan_step",
                     "norm", "norm", "norm_bwd"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("conv", "conv_bwd"):
        B = rng.choice([1, 1, 2, 3])
        D = _log_int(rng, 64, 4096)
        T = _log_int(rng, 1, 16384 * 1024 // (D * B))
        T = max(1, min(T, 16384) if kind == "bf16" else min(T, 8192))
        seqs = rng.choice([0, 0, 1, 2, 5, 9]) if B == 1 else 0
        return dict(op=op, type=kind, B=B, T=T, D=D, W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7, seqs=seqs,
                    bias=rng.random() < 0.5)
    if op == "conv_step":
        rows = _log_int(rng, 1, 256)
        return dict(op=op, type=kind, rows=rows, slots=rows + rng.randrange(64), D=_log_int(rng, 64, 8192),
                    W=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.7)
    if op in ("scan", "scan_bwd"):
        B = rng.choice([1, 1, 2])
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4])
        N, P = rng.choice([32, 64, 96, 128]), rng.choice([32, 64, 64, 128])
        top = 8192 * 32 * 128 * 128 // (B * H * N * P)
        T = _log_int(rng, 1, max(1, min(top, 8192 if kind == "bf16" else 2048)))
        return dict(op=op, type=kind, B=B, T=T, H=H, G=G, N=N, P=P, seqs=rng.choice([0, 0, 1, 3, 7]) if B == 1 else 0)
    if op == "scan_step":
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4])
        rows = _log_int(rng, 1, 64)
        return dict(op=op, type=kind, rows=rows, slots=rows + rng.randrange(16), H=H, G=G,
                    N=rng.choice([32, 64, 96, 128]), P=rng.choice([32, 64, 64, 128]))
    D = _log_int(rng, 64, 8192)
    if rng.random() < 0.7:
        D = max(64, D // 64 * 64)
    rows = _log_int(rng, 1, 8192 * 4096 // D // (1 if kind == "bf16" else 2))
    if op == "norm_bwd":
        return dict(op=op, type=kind, rows=rows, D=D, residual=rng.random() < 0.7)
    quant = rng.choice([-1, 0, 128])
    return dict(op=op, type=kind, rows=rows, D=D, quant=quant if D % 128 == 0 or quant <= 0 else 0,
                residual=rng.random() < 0.7)


# ---------------------------------------------------------------------------------------------- inputs
def _offsets(case, gen):
    """Offsets of the packed sequences: ragged lengths, whole numbers from the seed, some of one token or none."""
    T, n = case["T"], case["seqs"]
    if not n:
        return None
    cuts = torch.randint(0, T + 1, (n - 1,), generator=gen).sort().values.tolist()
    return [0] + cuts + [T]


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = TYPES[case["type"]]
    op = case["op"]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=DEV) * (hi - lo) + lo

    s = dict(case=case)
    if op.startswith("conv"):
        D, W = case["D"], case["W"]
        s["weight"] = normal(D, W, std=W ** -0.5, dtype=torch.float32)
        s["bias"] = normal(D, std=0.2, dtype=torch.float32) if case.get("bias", True) else None
        s["act"] = "silu" if case["silu"] else None
    if op.startswith("scan"):
        H, G, N, P = case["H"], case["G"], case["N"], case["P"]
        # steps between 1e-3 and 0.1 after the softplus, decays from exp(-1) to exp(-16) for each unit of step
        s["A_log"] = uniform(1.0, 16.0, H).log()
        step = torch.exp(uniform(math.log(1e-3), math.log(0.1), H))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = uniform(0.5, 1.5, H)
    if op in ("conv", "conv_bwd"):
        B, T = case["B"], case["T"]
        s["x"] = normal(B, T, D)
        cu = _offsets(case, host)
        n = B if cu is None else len(cu) - 1
        s["h0"] = normal(n, W - 1, D)
    elif op == "conv_step":
        s["x"] = normal(case["rows"], D)
        s["state"] = normal(case["slots"], W - 1, D)
    elif op in ("scan", "scan_bwd"):
        B, T = case["B"], case["T"]
        s["x"], s["dt"] = normal(B, T, H, P), normal(B, T, H)
        s["B"], s["C"] = normal(B, T, G, N, std=N ** -0.25), normal(B, T, G, N, std=N ** -0.25)
        cu = _offsets(case, host)
        n = B if cu is None else len(cu) - 1
        s["h0"] = normal(n, H, N, P, std=0.3, dtype=torch.float32)
    elif op == "scan_step":
        R = case["rows"]
        s["x"], s["dt"] = normal(R, H, P), normal(R, H)
        s["B"], s["C"] = normal(R, G, N, std=N ** -0.25), normal(R, G, N, std=N ** -0.25)
        s["state"] = normal(case["slots"], H, N, P, std=0.3, dtype=torch.float32)
    elif op in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        s["weight"] = uniform(0.5, 1.5, D)
        s["x"] = normal(R, D)
        s["residual"] = normal(R, D, std=3.0) if case["residual"] else None
    if op in ("conv", "conv_bwd", "scan", "scan_bwd"):
        s["cu"] = cu
        s["cu_host"] = None if cu is None else torch.tensor(cu, dtype=torch.int64)
        s["cu_dev"] = None if cu is None else s["cu_host"].to(DEV)
    if op in ("conv_step", "scan_step"):
        s["slots"] = torch.randperm(case["slots"], generator=host)[:case["rows"]].to(torch.int32).to(DEV)
    if op == "conv_bwd":
        s["dy"], s["dht"] = normal(*s["x"].shape), normal(*s["h0"].shape)
    if op == "scan_bwd":
        s["dy"], s["dht"] = normal(*s["x"].shape), normal(*s["h0"].shape, std=0.3, dtype=torch.float32)
    if op == "norm_bwd":
        s["dy"] = normal(R, D)
    return s


# ---------------------------------------------------------------------------------------- the plain forms
def _softplus(v):
    return torch.clamp(v, min=0) + torch.log(1 + torch.exp(-torch.abs(v)))


def _positions(s):
    """Of each token: its sequence and its place in it; of each sequence: its start and length (tokens in one row)."""
    B, T = s["x"].shape[:2]
    cu = torch.arange(B + 1, device=DEV) * T if s["cu_dev"] is None else s["cu_dev"]
    t = torch.arange(B * T, device=DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, t - cu[seq], cu[:-1], cu[1:] - cu[:-1]


def _earlier(x, h0, seq, pos, k):
    """Each token's input k places earlier in its sequence, from the initial state where that lies before it."""
    if k == 0:
        return x
    back = torch.cat([x.new_zeros(min(k, len(x)), x.shape[1]), x[:max(0, len(x) - k)]])
    row = (pos - k + h0.shape[1]).clamp(0, h0.shape[1] - 1)
    return torch.where((pos >= k)[:, None], back, h0[seq, row])


def _conv_pre(s):
    W, D = s["weight"].shape[1], s["x"].shape[-1]
    x, h0 = s["x"].float().reshape(-1, D), s["h0"].float()
    seq, pos, start, length = _positions(s)
    pre = torch.zeros_like(x) if s["bias"] is None else s["bias"].expand_as(x).clone()
    for k in range(W):
        pre += s["weight"][:, W - 1 - k] * _earlier(x, h0, seq, pos, k)
    return x, h0, seq, pos, start, length, pre


def _conv(s):
    W, t = s["weight"].shape[1], s["x"].dtype
    x, h0, seq, pos, start, length, pre = _conv_pre(s)
    y = pre / (1 + torch.exp(-pre)) if s["act"] else pre
    p = length[:, None] - (W - 1) + torch.arange(W - 1, device=DEV)  # the places that the final state holds
    last = torch.where((p >= 0)[..., None], x[(start[:, None] + p).clamp(0, len(x) - 1)],
                       torch.gather(h0, 1, (p + W - 1).clamp(0, W - 2)[..., None].expand_as(h0)))
    return y.reshape(s["x"].shape).to(t), last.to(t)


def _conv_bwd(s):
    W, t = s["weight"].shape[1], s["x"].dtype
    x, h0, seq, pos, start, length, pre = _conv_pre(s)
    dpre = s["dy"].float().reshape(x.shape)
    if s["act"]:
        g = 1 / (1 + torch.exp(-pre))
        dpre = dpre * g * (1 + pre * (1 - g))
    left = length[seq] - 1 - pos
    dx, dw, dh0 = torch.zeros_like(x), torch.zeros_like(s["weight"]), torch.zeros_like(h0)
    for k in range(W):
        dw[:, W - 1 - k] = (dpre * _earlier(x, h0, seq, pos, k)).sum(0)
        ahead = torch.cat([dpre[min(k, len(x)):], dpre.new_zeros(min(k, len(x)), x.shape[1])])
        dx += s["weight"][:, W - 1 - k] * torch.where((left >= k)[:, None], ahead, 0)
        for r in range(W - 1):
            q = r - (W - 1) + k  # the place whose output reads row r with this weight
            if q >= 0:
                there = dpre[(start + q).clamp(max=len(x) - 1)]
                dh0[:, r] += s["weight"][:, W - 1 - k] * torch.where((length > q)[:, None], there, 0)
    for r in range(W - 1):
        p = length - (W - 1) + r
        at = (start + p).clamp(0, len(x) - 1)
        dx.index_add_(0, at, torch.where((p >= 0)[:, None], s["dht"][:, r].float(), 0))
        for n in range(W - 1):
            dh0[:, n] += torch.where((p + W - 1 == n)[:, None], s["dht"][:, r].float(), 0)
    out = dict(dx=dx.reshape(s["x"].shape).to(t), dweight=dw, dh0=dh0.to(t))
    if s["bias"] is not None:
        out["dbias"] = dpre.sum(0)
    return out


def _conv_step(s):
    W, t = s["weight"].shape[1], s["x"].dtype
    at = s["slots"].long()
    window = torch.cat([s["state"][at], s["x"][:, None]], 1)
    pre = (window.float() * s["weight"].t()).sum(1) + s["bias"]
    y = pre / (1 + torch.exp(-pre)) if s["act"] else pre
    s["state"][at] = window[:, 1:]
    return y.to(t), s["state"]


def _scan_rows(x, d, A, Bm, C, D, h0):
    """The scan of a batch of rows of one length: chunks of products, and a product over the chunks for the states."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    pad = -T % CHUNK

    def cut(v):  # [B, T, heads, n] -> [B, heads, chunks, CHUNK, n]
        v = torch.cat([v, v.new_zeros(B, pad, *v.shape[2:])], 1) if pad else v
        return v.reshape(B, -1, CHUNK, *v.shape[2:]).permute(0, 3, 1, 2, 4)

    Bc, Cc = cut(Bm).repeat_interleave(H // G, 1), cut(C).repeat_interleave(H // G, 1)
    u = cut(x * d[..., None])
    cum = cut((d.double() * A.double())[..., None])[..., 0].cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf)).float()
    y = (Cc @ Bc.transpose(-1, -2) * decay) @ u
    states = (Bc * torch.exp(cum[..., -1:] - cum).float()[..., None]).transpose(-1, -2) @ u
    states = torch.cat([h0[:, :, None], states], 2)
    ends = torch.cat([cum.new_zeros(B, H, 1), cum[..., -1].cumsum(-1)], -1)
    low = torch.ones(ends.shape[-1], ends.shape[-1], dtype=torch.bool, device=x.device).tril()
    pass_on = torch.exp((ends[..., :, None] - ends[..., None, :]).masked_fill(~low, -math.inf)).float()
    states = (pass_on @ states.flatten(3)).reshape(states.shape)
    y = y + torch.exp(cum).float()[..., None] * (Cc @ states[:, :, :-1])
    y = y.permute(0, 2, 3, 1, 4).reshape(B, T + pad, H, P)[:, :T]
    return y + D[:, None] * x, states[:, :, -1]


def _scan_plain(x, dt, A_log, Bm, C, D, dt_bias, h0, cu):
    d, A = _softplus(dt + dt_bias), -torch.exp(A_log)
    if cu is None:
        return _scan_rows(x, d, A, Bm, C, D, h0)
    parts = [_scan_rows(x[:, a:b], d[:, a:b], A, Bm[:, a:b], C[:, a:b], D, h0[n:n + 1]) if a < b else (x[:, a:b], h0[n:n + 1])
             for n, (a, b) in enumerate(zip(cu, cu[1:]))]
    return torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts])


def _scan(s):
    y, last = _scan_plain(s["x"].float(), s["dt"].float(), s["A_log"], s["B"].float(), s["C"].float(), s["D"],
                          s["dt_bias"], s["h0"], s["cu"])
    return y.to(s["x"].dtype), last


GRADS = dict(x="dx", dt="ddt", A_log="dA_log", B="dB", C="dC", D="dD", dt_bias="ddt_bias", h0="dh0")


def _scan_bwd(s):
    leaves = {k: s[k].float().detach().clone().requires_grad_() for k in GRADS}
    y, last = _scan_plain(leaves["x"], leaves["dt"], leaves["A_log"], leaves["B"], leaves["C"], leaves["D"],
                          leaves["dt_bias"], leaves["h0"], s["cu"])
    grads = torch.autograd.grad([y, last], list(leaves.values()), [s["dy"].float(), s["dht"]])
    return {GRADS[k]: g.to(s[k].dtype) for k, g in zip(leaves, grads)}


def _scan_step(s):
    H, G = s["x"].shape[1], s["B"].shape[1]
    at = s["slots"].long()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(-torch.exp(s["A_log"]) * d)
    Bm, C = (s[k].float().repeat_interleave(H // G, 1) for k in ("B", "C"))
    x = s["x"].float()
    state = a[..., None, None] * s["state"][at] + Bm[..., None] * (d[..., None] * x)[:, :, None]
    s["state"][at] = state
    y = (state * C[..., None]).sum(2) + s["D"][:, None] * x
    return y.to(s["x"].dtype), s["state"]


def _norm(s):
    t, D = s["x"].dtype, s["x"].shape[1]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(t)
    f = h.float()
    y = f / torch.sqrt((f * f).mean(1, keepdim=True) + 1e-6) * s["weight"]
    quant = s["case"]["quant"]
    if quant < 0:
        return y.to(t), h
    y = y.reshape(len(y), -1, quant or D)
    scale = y.abs().amax(2).clamp(min=1e-30) / 448
    q = (y / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(-1, D), scale, h


def _norm_bwd(s):
    h, w, dy = s["x"].float(), s["weight"], s["dy"].float()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)
    g = dy * w
    dx = r * g - h * r ** 3 * (g * h).mean(1, keepdim=True)
    if s["residual"] is not None:
        dx = dx + s["residual"].float()  # the gradient that arrives at the residual
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * h * r).sum(0))


PLAIN = dict(conv=_conv, conv_bwd=_conv_bwd, conv_step=_conv_step, scan=_scan, scan_bwd=_scan_bwd,
             scan_step=_scan_step, norm=_norm, norm_bwd=_norm_bwd)


# ------------------------------------------------------------------------------ this package's entry points
def _own_run(s):
    import gated_delta_rule_log2_amd as kda
    op = s["case"]["op"]
    if op.startswith("conv"):
        args = dict(bias=s["bias"], activation=s["act"])
        if op == "conv_step":
            return kda.short_conv_step(s["x"], s["state"], s["weight"], slots=s["slots"], **args), s["state"]
        args.update(initial_state=s["h0"], cu_seqlens=s["cu_dev"], cu_seqlens_host=s["cu_host"])
        if op == "conv":
            return kda.short_conv(s["x"], s["weight"], output_final_state=True, **args)
        return kda.short_conv_bwd(s["x"], s["weight"], s["dy"], dht=s["dht"], **args)
    if op.startswith("scan"):
        args = dict(D=s["D"], dt_bias=s["dt_bias"], use_softplus_in_kernel=True)
        inputs = [s[k] for k in ("x", "dt", "A_log", "B", "C")]
        if op == "scan_step":
            return kda.ssm_step(*inputs, s["state"], slots=s["slots"], **args), s["state"]
        args.update(initial_state=s["h0"], cu_seqlens=s["cu_dev"], cu_seqlens_host=s["cu_host"])
        if op == "scan":
            return kda.chunk_ssm(*inputs, output_final_state=True, **args)
        return kda.chunk_ssm_bwd(*inputs, s["dy"], dht=s["dht"], **args)
    if op == "norm_bwd":
        return kda.rms_norm_bwd(s["x"], s["weight"], s["dy"], dh=s["residual"], eps=1e-6)
    if s["case"]["quant"] < 0:
        return kda.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6)
    return kda.rms_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=1e-6, group_size=s["case"]["quant"])


def run(state):
    return _own_run(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------- the definitions in 64 bits
def _sequences(s):
    """(row of the batch, first token, last token) of each sequence."""
    B, T = s["x"].shape[:2]
    if s["cu"] is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, a, b) for a, b in zip(s["cu"], s["cu"][1:])]


def _exact_conv(s):
    op, w = s["case"]["op"], s["weight"].double()
    W, x = w.shape[1], s["x"].double()

    def output(window, n):  # of n tokens whose inputs, with those before them, are `window`
        pre = window.unfold(0, W, 1)[:n].mul(w).sum(-1) if n else window[:0]
        return pre + (0 if s["bias"] is None else s["bias"].double())

    if op == "conv_step":
        state = s["state"].double()
        at = s["slots"].long()
        window = torch.cat([state[at], x[:, None]], 1)
        pre = torch.einsum("rwd,dw->rd", window, w) + s["bias"].double()
        state[at] = window[:, 1:]
        return (pre * torch.sigmoid(pre) if s["act"] else pre), state
    y, last = torch.zeros_like(x), s["h0"].double().clone()
    dx, dw, db, dh0 = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(w[:, 0]), torch.zeros_like(last)
    for n, (r, a, b) in enumerate(_sequences(s)):
        window = torch.cat([s["h0"][n].double(), x[r, a:b]])
        pre = output(window, b - a)
        if op == "conv":
            y[r, a:b] = pre * torch.sigmoid(pre) if s["act"] else pre
            last[n] = window[b - a:]
            continue
        dpre = s["dy"][r, a:b].double()
        if s["act"]:
            g = torch.sigmoid(pre)
            dpre = dpre * (g + pre * g * (1 - g))
        dwindow = torch.zeros_like(window)
        dwindow[b - a:] += s["dht"][n].double()
        for k in range(W):
            dwindow[k:k + b - a] += w[:, k] * dpre
            dw[:, k] += (dpre * window[k:k + b - a]).sum(0)
        db += dpre.sum(0)
        dh0[n], dx[r, a:b] = dwindow[:W - 1], dwindow[W - 1:]
    if op == "conv":
        return y, last
    return dict(dx=dx, dweight=dw, dh0=dh0, **({} if s["bias"] is None else dict(dbias=db)))


def _exact_scan(s):
    op = s["case"]["op"]
    H, G = s["x"].shape[-2], s["B"].shape[-2]
    raw = s["dt"].double() + s["dt_bias"].double()
    d, A = torch.log1p(torch.exp(raw)), -torch.exp(s["A_log"].double())
    a = torch.exp(d * A)
    x, D = s["x"].double(), s["D"].double()
    Bm, C = (s[k].double().repeat_interleave(H // G, -2) for k in ("B", "C"))
    if op == "scan_step":
        state, at = s["state"].double(), s["slots"].long()
        state[at] = a[..., None, None] * state[at] + torch.einsum("rh,rhn,rhp->rhnp", d, Bm, x)
        return torch.einsum("rhnp,rhn->rhp", state[at], C) + D[:, None] * x, state
    y, last = torch.zeros_like(x), s["h0"].double().clone()
    rows = [(slice(None), slice(None), 0, x.shape[1])] if s["cu"] is None else [
        (slice(0, 1), slice(n, n + 1), p, q) for n, (_, p, q) in enumerate(_sequences(s))]
    if op == "scan":
        for r, n, p, q in rows:
            S = s["h0"][n].double().clone()
            for t in range(p, q):
                S.mul_(a[r, t, :, None, None]).add_((d[r, t, :, None] * Bm[r, t])[..., None] * x[r, t][:, :, None])
                y[r, t] = (S * C[r, t][..., None]).sum(2)
            last[n] = S
        return y + D[:, None] * x, last
    dy = s["dy"].double()
    dx, dB, dC, dd, da = (torch.zeros_like(v) for v in (x, Bm, C, d, d))
    dh0 = torch.zeros_like(last)
    for r, n, p, q in rows:
        S = torch.empty(q - p + 1, *s["h0"][n].shape, dtype=torch.float64, device=x.device)
        S[0] = s["h0"][n]
        for t in range(p, q):
            torch.mul(S[t - p], a[r, t, :, None, None], out=S[t - p + 1])
            S[t - p + 1].add_((d[r, t, :, None] * Bm[r, t])[..., None] * x[r, t][:, :, None])
        R = s["dht"][n].double().clone()
        for t in range(q - 1, p - 1, -1):
            R.add_(C[r, t][..., None] * dy[r, t][:, :, None])
            dC[r, t] = (S[t - p + 1] * dy[r, t][:, :, None]).sum(-1)
            Rx, RB = (R * x[r, t][:, :, None]).sum(-1), (R * Bm[r, t][..., None]).sum(2)
            dB[r, t] = d[r, t][..., None] * Rx
            dx[r, t] = d[r, t][..., None] * RB
            dd[r, t] = (Rx * Bm[r, t]).sum(-1)
            da[r, t] = (R * S[t - p]).sum((-1, -2))
            R.mul_(a[r, t, :, None, None])
        dh0[n] = R
        del S
    dl = da * a  # by the logarithm of the decay, d * A
    dd = (dd + dl * A) * torch.sigmoid(raw)
    group = (*s["B"].shape[:3], H // G, -1)
    return dict(dx=dx + D[:, None] * dy, ddt=dd, dA_log=(dl * d * A).sum((0, 1)), dh0=dh0,
                dB=dB.reshape(*s["B"].shape[:3], H // G, -1).sum(3), dC=dC.reshape(group).sum(3),
                dD=(dy * x).sum((0, 1, 3)), ddt_bias=dd.sum((0, 1)))


def _exact_norm(s):
    if s["case"]["op"] == "norm_bwd":
        h, w, dy = s["x"].double(), s["weight"].double(), s["dy"].double()
        unit = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        g = dy * w
        dx = (g - unit * (g * unit).mean(1, keepdim=True)) * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        return dict(dx=dx + (0 if s["residual"] is None else s["residual"].double()), dweight=(dy * unit).sum(0))
    h = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
    y = h.double() * (h.double().square().mean(1, keepdim=True) + 1e-6).rsqrt() * s["weight"].double()
    quant = s["case"]["quant"]
    if quant < 0:
        return y, h.double()
    y = y.reshape(len(y), -1, quant or h.shape[1])
    scale = y.abs().amax(2) / 448
    return (y / scale[..., None]).reshape(h.shape), scale, h.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_conv(s) if op.startswith("conv") else _exact_scan(s) if op.startswith("scan") else _exact_norm(s)


# --------------------------------------------------------------------------------------------- what it costs
def work(case):
    """Each input read once and each output written once; the operations of the token-by-token form."""
    e = 2 if case["type"] == "bf16" else 4
    op = case["op"]
    if op in ("conv", "conv_bwd"):
        D, W, tokens = case["D"], case["W"], case["B"] * case["T"]
        states = (case["seqs"] or case["B"]) * (W - 1) * D * e
        few = (W + 1) * D * 4
        if op == "conv":
            return dict(bytes=2 * tokens * D * e + 2 * states + few, flops=tokens * D * (2 * W + 5 * case["silu"]))
        return dict(bytes=3 * tokens * D * e + 3 * states + 2 * few, flops=tokens * D * (6 * W + 10 * case["silu"]))
    if op == "conv_step":
        D, W, rows = case["D"], case["W"], case["rows"]
        return dict(bytes=rows * D * e * 2 * W + (W + 1) * D * 4, flops=rows * D * (2 * W + 5 * case["silu"]))
    if op.startswith("scan"):
        H, G, N, P = case["H"], case["G"], case["N"], case["P"]
        tokens = case["rows"] if op == "scan_step" else case["B"] * case["T"]
        seqs = case["rows"] if op == "scan_step" else case["seqs"] or case["B"]
        heads, groups, state = tokens * H * (P + 0.5) * e, tokens * G * N * e, seqs * H * N * P * 4
        if op == "scan_bwd":  # x, dt, B, C, dy in, their gradients out; the states' and what arrives at them
            return dict(bytes=3 * heads + tokens * H * 0.5 * e + 4 * groups + 3 * state, flops=tokens * H * N * P * 14)
        return dict(bytes=2 * heads + 2 * groups + 2 * state, flops=tokens * H * N * P * 5)
    rows, D = case["rows"], case["D"]
    values = rows * D
    if op == "norm_bwd":
        return dict(bytes=values * e * (3 + case["residual"]) + 8 * D, flops=values * 9)
    scales = 0 if case["quant"] < 0 else rows * (D // case["quant"] if case["quant"] else 1) * 4
    out = e if case["quant"] < 0 else 1
    return dict(bytes=values * (e * (1 + 2 * case["residual"]) + out) + scales + 4 * D, flops=values * 6)
