"""Refusals of the layer operators' C entries and of their Python functions (no GPU: every
check runs on the host before any HIP call)."""
import ctypes

import pytest
import torch

import gated_delta_rule_log2_amd as kda
from gated_delta_rule_log2_amd import _abi

S = _abi.STATUS
FAKE = 0x1000  # never dereferenced
BF16, FP32 = _abi.DTYPE_BF16, _abi.DTYPE_FP32


@pytest.fixture(scope="module")
def lib():
    return _abi.load_library()


def offsets(vals):
    arr = (ctypes.c_int64 * len(vals))(*vals)
    return arr, ctypes.cast(arr, ctypes.POINTER(ctypes.c_int64))


def conv_desc(**kw):
    d = _abi.KdaConvDesc()
    for k, v in dict(dict(B=1, T=64, D=128, W=4, num_seqs=1, x_dtype=BF16, w_dtype=FP32, dy_dtype=BF16, flags=1,
                          x_stride=128), **kw).items():
        setattr(d, k, v)
    return d


def conv_calls(lib, d, p=FAKE, cu=None, ws=FAKE, nbytes=1 << 40, h0=None):
    r = ctypes.byref(d)
    return (lib.kda_short_conv_fwd(r, p, p, None, h0, cu, p, None, None),
            lib.kda_short_conv_bwd(r, p, p, None, h0, cu, p, None, p, p, None, None, ws, nbytes, None))


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(D=0), "SHAPE"), (dict(W=0), "SHAPE"), (dict(num_seqs=2), "SHAPE"),
    (dict(x_stride=127), "SHAPE"), (dict(B=1 << 16, T=1 << 16, num_seqs=1 << 16), "SHAPE"),
    (dict(W=1), "UNSUPPORTED"), (dict(W=5), "UNSUPPORTED"), (dict(flags=2), "UNSUPPORTED"),
    (dict(x_dtype=2), "DTYPE"), (dict(w_dtype=-1), "DTYPE"), (dict(dy_dtype=9), "DTYPE"),
])
def test_conv_descriptor(lib, kw, code):
    assert set(conv_calls(lib, conv_desc(**kw))) == {S["KDA_ERR_" + code]}


def test_conv_pointers_and_workspace(lib):
    assert set(conv_calls(lib, conv_desc(), p=None)) == {S["KDA_ERR_NULL_POINTER"]}
    assert conv_calls(lib, conv_desc(), ws=None)[1] == S["KDA_ERR_WORKSPACE"]
    n = ctypes.c_size_t(0)
    assert lib.kda_short_conv_bwd_workspace_size(ctypes.byref(conv_desc()), ctypes.byref(n)) == 0 and n.value > 0
    assert conv_calls(lib, conv_desc(), nbytes=n.value - 1)[1] == S["KDA_ERR_WORKSPACE"]
    assert conv_calls(lib, conv_desc(x_dtype=FP32, dy_dtype=BF16))[1] == S["KDA_ERR_DTYPE"]
    assert lib.kda_short_conv_bwd_workspace_size(None, ctypes.byref(n)) == S["KDA_ERR_NULL_POINTER"]
    d = conv_desc()
    assert lib.kda_short_conv_fwd(ctypes.byref(d), FAKE, FAKE, None, FAKE, None, FAKE, FAKE, None) == S["KDA_ERR_UNSUPPORTED"]


@pytest.mark.parametrize("vals,B,T", [([1, 64], 1, 64), ([0, 63], 1, 64), ([0, 40, 20, 64], 1, 64), ([0, 32, 64], 2, 32)])
def test_conv_offsets(lib, vals, B, T):
    arr, ptr = offsets(vals)
    d = conv_desc(B=B, T=T, num_seqs=len(vals) - 1, cu_seqlens_host=ptr)
    assert set(conv_calls(lib, d, cu=FAKE)) == {S["KDA_ERR_VARLEN"]}


def test_offsets_come_in_two_copies(lib):
    arr, ptr = offsets([0, 10, 64])
    assert set(conv_calls(lib, conv_desc(num_seqs=2, cu_seqlens_host=ptr))) == {S["KDA_ERR_VARLEN"]}
    assert set(conv_calls(lib, conv_desc(), cu=FAKE)) == {S["KDA_ERR_VARLEN"]}


def test_conv_step(lib):
    def call(d, slots=FAKE, pool=8, state=FAKE, p=FAKE):
        return lib.kda_short_conv_step(ctypes.byref(d), p, p, None, state, slots, pool, p, None)

    one = dict(B=4, T=1, num_seqs=4)
    assert call(conv_desc()) == S["KDA_ERR_SHAPE"]  # T = 64
    assert call(conv_desc(**one), slots=None, pool=3) == S["KDA_ERR_SHAPE"]
    assert call(conv_desc(**one), pool=-1) == S["KDA_ERR_SHAPE"]
    assert call(conv_desc(**one), state=None) == S["KDA_ERR_NULL_POINTER"]
    assert call(conv_desc(**one), p=None) == S["KDA_ERR_NULL_POINTER"]
    arr, ptr = offsets([0, 1])
    assert call(conv_desc(T=1, cu_seqlens_host=ptr)) == S["KDA_ERR_VARLEN"]


def norm_desc(**kw):
    d = _abi.KdaNormDesc()
    for k, v in dict(dict(rows=16, D=256, group_size=0, x_dtype=BF16, w_dtype=FP32, eps=1e-6), **kw).items():
        setattr(d, k, v)
    return d


def norm_calls(lib, d, p=FAKE, ws=FAKE, nbytes=1 << 40):
    r = ctypes.byref(d)
    return (lib.kda_rms_norm_fwd(r, p, None, p, p, None, None), lib.kda_rms_norm_fp8(r, p, None, p, p, p, None, None),
            lib.kda_rms_norm_bwd(r, p, p, p, None, p, p, ws, nbytes, None))


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "SHAPE"), (dict(D=0), "SHAPE"), (dict(group_size=-8), "SHAPE"), (dict(eps=float("nan")), "SHAPE"),
    (dict(eps=-1.0), "SHAPE"), (dict(rows=1 << 31), "SHAPE"), (dict(D=32769), "UNSUPPORTED"),
    (dict(x_dtype=5), "DTYPE"), (dict(w_dtype=5), "DTYPE"),
])
def test_norm_descriptor(lib, kw, code):
    assert set(norm_calls(lib, norm_desc(**kw))) == {S["KDA_ERR_" + code]}


@pytest.mark.parametrize("group,D", [(4, 256), (24, 240), (1024, 4096), (128, 192)])
def test_norm_groups(lib, group, D):
    assert norm_calls(lib, norm_desc(group_size=group, D=D))[1] == S["KDA_ERR_UNSUPPORTED"]


def test_norm_pointers_and_workspace(lib):
    assert set(norm_calls(lib, norm_desc(), p=None)) == {S["KDA_ERR_NULL_POINTER"]}
    assert norm_calls(lib, norm_desc(), ws=None)[2] == S["KDA_ERR_WORKSPACE"]
    n = ctypes.c_size_t(0)
    assert lib.kda_rms_norm_bwd_workspace_size(ctypes.byref(norm_desc()), ctypes.byref(n)) == 0
    assert norm_calls(lib, norm_desc(), nbytes=n.value - 1)[2] == S["KDA_ERR_WORKSPACE"]


X, WGT = torch.zeros(2, 5, 16), torch.zeros(16, 4)


@pytest.mark.parametrize("call", [
    lambda: kda.short_conv(X[0], WGT), lambda: kda.short_conv(X, torch.zeros(16, 5)),
    lambda: kda.short_conv(X[:0], WGT), lambda: kda.short_conv_step(X, X, WGT),
    lambda: kda.short_conv_bwd(X, torch.zeros(16), X),
])
def test_python_refuses(call):
    with pytest.raises(kda.KDAContractError):
        call()


@pytest.mark.parametrize("call", [
    lambda: kda.short_conv(X, WGT), lambda: kda.short_conv_bwd(X, WGT, X), lambda: kda.short_conv_step(X[0], X, WGT),
    lambda: kda.rms_norm(X, X[0, 0]), lambda: kda.rms_norm_fp8(X, X[0, 0]), lambda: kda.rms_norm_bwd(X, X[0, 0], X),
])
def test_python_refuses_cpu_tensors(call):
    with pytest.raises(kda.KDARuntimeError):
        call()


def ssm_desc(**kw):
    d = _abi.KdaSsmDesc()
    for k, v in dict(dict(B=1, T=64, H=4, G=2, N=64, P=64, num_seqs=1, x_dtype=BF16, dt_dtype=FP32, flags=1, x_stride=256,
                          dt_stride=4, b_stride=128, c_stride=128), **kw).items():
        setattr(d, k, v)
    return d


def ssm_calls(lib, d, p=FAKE, A=FAKE, cu=None, ws=FAKE, nbytes=1 << 40, h0=None, ht=None):
    r = ctypes.byref(d)
    return (lib.kda_ssm_fwd(r, p, p, A, p, p, None, None, h0, cu, p, ht, ws, nbytes, None),
            lib.kda_ssm_bwd(r, p, p, A, p, p, None, None, h0, cu, p, None, p, p, FAKE, p, p, None, None, None, ws, nbytes, None))


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(G=0), "SHAPE"), (dict(num_seqs=3), "SHAPE"),
    (dict(x_stride=255), "SHAPE"), (dict(dt_stride=3), "SHAPE"), (dict(b_stride=127), "SHAPE"), (dict(c_stride=127), "SHAPE"),
    (dict(B=1 << 15, T=1 << 16, num_seqs=1 << 15), "SHAPE"), (dict(G=3), "GVA"), (dict(N=48), "UNSUPPORTED"),
    (dict(N=160, b_stride=320, c_stride=320), "UNSUPPORTED"), (dict(P=16), "UNSUPPORTED"),
    (dict(P=256, x_stride=1024), "UNSUPPORTED"), (dict(flags=2), "UNSUPPORTED"), (dict(x_dtype=2), "DTYPE"), (dict(dt_dtype=2), "DTYPE"),
])
def test_ssm_descriptor(lib, kw, code):
    assert set(ssm_calls(lib, ssm_desc(**kw))) == {S["KDA_ERR_" + code]}


def test_ssm_pointers_and_workspace(lib):
    assert set(ssm_calls(lib, ssm_desc(), p=None)) == {S["KDA_ERR_NULL_POINTER"]}
    assert set(ssm_calls(lib, ssm_desc(), A=None)) == {S["KDA_ERR_MISSING_A_LOG"]}
    assert set(ssm_calls(lib, ssm_desc(), cu=FAKE)) == {S["KDA_ERR_VARLEN"]}
    assert ssm_calls(lib, ssm_desc(), h0=FAKE, ht=FAKE)[0] == S["KDA_ERR_UNSUPPORTED"]
    for i, size in enumerate((lib.kda_ssm_fwd_workspace_size, lib.kda_ssm_bwd_workspace_size)):
        n = ctypes.c_size_t(0)
        assert size(ctypes.byref(ssm_desc()), ctypes.byref(n)) == 0 and n.value > 0
        assert ssm_calls(lib, ssm_desc(), nbytes=n.value - 1)[i] == S["KDA_ERR_WORKSPACE"]
        assert ssm_calls(lib, ssm_desc(), ws=None)[i] == S["KDA_ERR_WORKSPACE"]
        assert size(None, ctypes.byref(n)) == S["KDA_ERR_NULL_POINTER"]
        assert size(ctypes.byref(ssm_desc()), None) == S["KDA_ERR_NULL_POINTER"]
        assert size(ctypes.byref(ssm_desc(T=0)), ctypes.byref(n)) == 0


@pytest.mark.parametrize("vals,B,T", [([1, 64], 1, 64), ([0, 63], 1, 64), ([0, 40, 20, 64], 1, 64), ([0, 32, 64], 2, 32)])
def test_ssm_offsets(lib, vals, B, T):
    arr, ptr = offsets(vals)
    assert set(ssm_calls(lib, ssm_desc(B=B, T=T, num_seqs=len(vals) - 1, cu_seqlens_host=ptr), cu=FAKE)) == {S["KDA_ERR_VARLEN"]}


def test_ssm_step(lib):
    def call(d, slots=FAKE, pool=8, state=FAKE, p=FAKE, A=FAKE):
        return lib.kda_ssm_step(ctypes.byref(d), p, p, A, p, p, None, None, state, slots, pool, p, None)

    one = dict(B=4, T=1, num_seqs=4)
    assert call(ssm_desc()) == S["KDA_ERR_SHAPE"]
    assert call(ssm_desc(**one), slots=None, pool=3) == S["KDA_ERR_SHAPE"]
    assert call(ssm_desc(**one), state=None) == S["KDA_ERR_NULL_POINTER"]
    assert call(ssm_desc(**one), p=None) == S["KDA_ERR_NULL_POINTER"]
    assert call(ssm_desc(**one), A=None) == S["KDA_ERR_MISSING_A_LOG"]
    arr, ptr = offsets([0, 1])
    assert call(ssm_desc(T=1, cu_seqlens_host=ptr)) == S["KDA_ERR_VARLEN"]


def test_ssm_workspace_covers_every_split(lib):
    """Long and short, packed and not: sizes grow with the work and never overflow."""
    sizes = []
    for T in (1, 64, 8192, 1 << 20):
        n = ctypes.c_size_t(0)
        assert lib.kda_ssm_bwd_workspace_size(ctypes.byref(ssm_desc(T=T)), ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[-1] > (1 << 20) * 4 * 4 * 7  # seven fp32 values a token and head at least
    n = ctypes.c_size_t(0)
    huge = ssm_desc(T=1 << 30, H=1 << 12, x_stride=1 << 18, dt_stride=1 << 12)
    assert lib.kda_ssm_bwd_workspace_size(ctypes.byref(huge), ctypes.byref(n)) == S["KDA_ERR_SHAPE"]


X4, DT3, A1, B4 = torch.zeros(2, 5, 2, 32), torch.zeros(2, 5, 2), torch.zeros(2), torch.zeros(2, 5, 1, 32)


@pytest.mark.parametrize("call", [
    lambda: kda.chunk_ssm(X4[0], DT3, A1, B4, B4), lambda: kda.chunk_ssm(X4, DT3[..., None], A1, B4, B4),
    lambda: kda.chunk_ssm(X4[:, :, :0], DT3[..., :0], A1, B4, B4), lambda: kda.ssm_step(X4, DT3, A1, B4, B4, X4),
])
def test_python_refuses_ssm(call):
    with pytest.raises(kda.KDAContractError):
        call()


@pytest.mark.parametrize("call", [
    lambda: kda.chunk_ssm(X4, DT3, A1, B4, B4), lambda: kda.chunk_ssm_bwd(X4, DT3, A1, B4, B4, X4),
    lambda: kda.ssm_step(X4[:, 0], DT3[:, 0], A1, B4[:, 0], B4[:, 0], X4),
])
def test_python_refuses_ssm_on_the_cpu(call):
    with pytest.raises(kda.KDARuntimeError):
        call()
