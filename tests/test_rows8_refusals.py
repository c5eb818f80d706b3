"""What the norm, the 8-bit products and the log probabilities refuse, before anything is launched (CPU)."""
import ctypes as C

import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv
from tree_speculative_decoding_array_gb300 import _abi

PTR = 0x1000
NAN, INF = float("nan"), float("inf")


def norm(**kw):
    a = dict(x=PTR, residual=PTR, weight=PTR, rows=2, H=256, dtype=tsv.BF16, eps=1e-6, offset=0.0, residual_out=PTR, out=PTR,
             out8=PTR, out8_scale=PTR)
    assert set(kw) <= set(a)
    return tsv.load().tsv_add_rms_norm(*{**a, **kw}.values(), None)


def quantize(**kw):
    a = dict(x=PTR, rows=2, H=256, dtype=tsv.BF16, out8=PTR, out8_scale=PTR)
    assert set(kw) <= set(a)
    return tsv.load().tsv_quantize_e4m3(*{**a, **kw}.values(), None)


def matmul(**kw):
    a = dict(a=PTR, a_scale=PTR, rows=2, K=256, w=PTR, w_scale=PTR, N=64, out=PTR, dtype=tsv.BF16)
    assert set(kw) <= set(a)
    return tsv.load().tsv_matmul_e4m3(*{**a, **kw}.values(), None)


def best(**kw):
    a = dict(a=PTR, a_scale=PTR, rows=2, K=256, w=PTR, w_scale=PTR, N=64, argmax=PTR, maxval=PTR, ws=PTR, ws_bytes=256)
    assert set(kw) <= set(a)
    return tsv.load().tsv_matmul_e4m3_argmax(*{**a, **kw}.values(), None)


def head(**kw):
    a = dict(hidden=PTR, rows=2, H=256, V=1000, dtype=tsv.E4M3_B128, W=PTR, scales=PTR, biases=None, argmax=PTR, maxlogit=PTR,
             ws=PTR, ws_bytes=1 << 20)
    assert set(kw) <= set(a)
    return tsv.load().tsv_lm_head_argmax(*{**a, **kw}.values(), None)


def logprobs(**kw):
    a = dict(logits=PTR, dtype=tsv.F32, rows=2, V=1000, targets=PTR, t=1.0, top_k=5, logp=PTR, rank=PTR, entropy=PTR, top_tokens=PTR,
             top_logp=PTR, ws=PTR, ws_bytes=1 << 24)
    assert set(kw) <= set(a)
    return tsv.load().tsv_token_logprobs(*{**a, **kw}.values(), None)


@pytest.fixture(autouse=True)
def no_error_left_behind():
    yield
    assert norm(rows=0) == _abi.OK  # a call that succeeds clears this thread's reason


@pytest.mark.parametrize("call, kw, status, word", [
    (norm, dict(rows=-1), "EINVAL", b"rows=-1"), (norm, dict(H=0), "EINVAL", b"H=0"), (norm, dict(H=32769), "ECAPACITY", b"32768"),
    (norm, dict(dtype=tsv.I8_SCALED), "EUNSUPPORTED", b"type 2"), (norm, dict(eps=0.0), "EINVAL", b"eps"), (norm, dict(eps=NAN), "EINVAL", b"eps"),
    (norm, dict(eps=INF), "EINVAL", b"eps"), (norm, dict(offset=NAN), "EINVAL", b"weight_offset"), (norm, dict(x=None), "EINVAL", b"null"),
    (norm, dict(weight=None), "EINVAL", b"null"), (norm, dict(out8=None), "EINVAL", b"together"), (norm, dict(out8_scale=None), "EINVAL", b"together"),
    (norm, dict(out=None, out8=None, out8_scale=None, residual_out=None), "EINVAL", b"no output"), (norm, dict(x=PTR + 1), "EINVAL", b"aligned"),
    (norm, dict(out8_scale=PTR + 2), "EINVAL", b"aligned"), (norm, dict(out=PTR + 2, dtype=tsv.F32), "EINVAL", b"aligned"),
    (quantize, dict(rows=-1), "EINVAL", b"rows"), (quantize, dict(H=0), "EINVAL", b"H=0"), (quantize, dict(dtype=7), "EUNSUPPORTED", b"type 7"),
    (quantize, dict(x=None), "EINVAL", b"null"), (quantize, dict(out8_scale=None), "EINVAL", b"null"), (quantize, dict(x=PTR + 1), "EINVAL", b"aligned"),
    (matmul, dict(rows=-1), "EINVAL", b"rows"), (matmul, dict(K=0), "EINVAL", b"K=0"), (matmul, dict(N=0), "EINVAL", b"N=0"),
    (matmul, dict(K=136), "EINVAL", b"multiple of 16"), (matmul, dict(dtype=tsv.I4_G64), "EUNSUPPORTED", b"output type"),
    (matmul, dict(a=PTR + 8), "EINVAL", b"16-byte"), (matmul, dict(w=PTR + 8), "EINVAL", b"16-byte"), (matmul, dict(a_scale=PTR + 2), "EINVAL", b"4-byte"),
    (matmul, dict(out=PTR + 1), "EINVAL", b"aligned"), (matmul, dict(out=None), "EINVAL", b"null"), (matmul, dict(w_scale=None), "EINVAL", b"null"),
    (matmul, dict(rows=(1 << 30) + 1), "ECAPACITY", b"2^30"), (matmul, dict(N=(1 << 30) + 1), "ECAPACITY", b"2^30"),
    (best, dict(K=8), "EINVAL", b"multiple of 16"), (best, dict(argmax=None), "EINVAL", b"null"), (best, dict(ws=None), "EINVAL", b"null"),
    (best, dict(ws=PTR + 8), "EINVAL", b"16-byte"), (best, dict(ws_bytes=255), "ECAPACITY", b"256"),
    (head, dict(H=264), "EINVAL", b"multiple of 16"), (head, dict(scales=None), "EINVAL", b"scales"), (head, dict(scales=PTR + 2), "EINVAL", b"4-byte"),
    (head, dict(W=PTR + 4), "EINVAL", b"16-byte"), (head, dict(ws=PTR + 8), "EINVAL", b"16-byte"), (head, dict(ws_bytes=512), "ECAPACITY", b"workspace"),
    (head, dict(dtype=tsv.F32), "EUNSUPPORTED", b"format 6"),
    (head, dict(rows=(1 << 30) + 1), "ECAPACITY", b"2^30"), (head, dict(V=(1 << 30) + 1), "ECAPACITY", b"2^30"),
    (logprobs, dict(rows=-1), "EINVAL", b"rows"), (logprobs, dict(V=0), "EINVAL", b"V=0"), (logprobs, dict(V=(1 << 24) + 1), "EINVAL", b"2^24"),
    (logprobs, dict(dtype=tsv.I8_SCALED), "EUNSUPPORTED", b"type 2"), (logprobs, dict(top_k=65), "EUNSUPPORTED", b"top_k=65"),
    (logprobs, dict(top_k=-1), "EUNSUPPORTED", b"top_k=-1"), (logprobs, dict(V=4), "EUNSUPPORTED", b"top_k=5"), (logprobs, dict(t=0.0), "EINVAL", b"temperature"),
    (logprobs, dict(t=NAN), "EINVAL", b"temperature"), (logprobs, dict(t=1e7), "EINVAL", b"temperature"), (logprobs, dict(logits=None), "EINVAL", b"null"),
    (logprobs, dict(targets=None), "EINVAL", b"together"), (logprobs, dict(logp=None), "EINVAL", b"together"),
    (logprobs, dict(targets=None, logp=None), "EINVAL", b"rank"), (logprobs, dict(top_tokens=None), "EINVAL", b"top_k=5"), (logprobs, dict(top_k=0), "EINVAL", b"top_k=0"),
    (logprobs, dict(targets=None, logp=None, rank=None, entropy=None, top_k=0, top_tokens=None, top_logp=None), "EINVAL", b"no output"),
    (logprobs, dict(logits=PTR + 2), "EINVAL", b"aligned"), (logprobs, dict(ws=None, V=100000), "EINVAL", b"workspace"), (logprobs, dict(ws=PTR + 8), "EINVAL", b"16-byte"),
    (logprobs, dict(ws_bytes=0, V=100000), "ECAPACITY", b"workspace"),
])
def test_refused(call, kw, status, word):
    assert call(**kw) == getattr(_abi, status)
    assert word in tsv.load().tsv_last_error()


def test_no_rows_are_no_work():
    for call in (norm, quantize, matmul, best, logprobs):
        assert call(rows=0) == _abi.OK
    lib = tsv.load()
    assert lib.tsv_matmul_e4m3_argmax_workspace_size(0) == 0 and lib.tsv_token_logprobs_workspace_size(0, 10, 1) == 0
    # the e4m3 head keeps the bests, the codes and the scales of its rows
    assert lib.tsv_lm_head_workspace_size(3, 272, 1000, tsv.E4M3_B128) == 256 + 1024 + 256


def test_the_binding_refuses():
    x, w = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tsv.add_rms_norm(x, w, eps=1e-6, out=x)
    with pytest.raises(ValueError, match="together"):
        tsv.add_rms_norm(x, w, eps=1e-6, out8=x)
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        tsv.quantize_e4m3(x.double(), x, x)
    with pytest.raises(ValueError, match="two dimensions"):
        tsv.add_rms_norm(w, w, eps=1e-6, out=w)
    with pytest.raises(ValueError, match="together"):
        tsv.token_logprobs(x, top_tokens=x)
    with pytest.raises(ValueError, match="no token"):
        tsv.token_logprobs(x, top_tokens=x[:, :0], top_logp=x[:, :0])
