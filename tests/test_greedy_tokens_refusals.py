"""What the step from likeliest tokens to greedy ones refuses, before anything is launched (CPU)."""
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv
from tree_speculative_decoding_array_gb300 import _abi

PTR = 0x1000


def greedy(**kw):
    a = dict(logits=PTR, rows=2, V=1000, top_tokens=PTR, top_k=5, argmax=PTR, maxlogit=PTR)
    assert set(kw) <= set(a)
    return tsv.load().tsv_greedy_tokens(*{**a, **kw}.values(), None)


@pytest.fixture(autouse=True)
def no_error_left_behind():
    yield
    assert greedy(rows=0) == _abi.OK


@pytest.mark.parametrize("kw, word", [
    (dict(rows=-1), b"rows=-1"), (dict(V=0), b"V=0"), (dict(V=(1 << 24) + 1), b"2^24"), (dict(top_k=0), b"top_k=0"), (dict(logits=None), b"null"),
    (dict(top_tokens=None), b"null"), (dict(argmax=None), b"null"), (dict(maxlogit=PTR + 2), b"aligned"), (dict(argmax=PTR + 1), b"aligned")])
def test_refused(kw, word):
    assert greedy(**kw) == _abi.EINVAL
    assert word in tsv.load().tsv_last_error()


def test_the_binding_refuses():
    x, i = torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tsv.greedy_tokens(x, i, i[:, 0].contiguous())
    with pytest.raises(ValueError, match="top_tokens"):
        tsv.greedy_tokens(x, i[:, :0], i[:, 0])
    with pytest.raises(ValueError, match="rows, V"):
        tsv.greedy_tokens(x[0], i, i[:, 0])
