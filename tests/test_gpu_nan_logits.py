"""A logit that is NaN, its sign bit clear, counts as larger than every number: its token wins, the lowest of several, and the largest logit is NaN."""
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
NAN = float("nan")


def spoiled(V):
    """Tokens whose logits are to be NaN: none in the first row's reach, the first two of a few that lie apart."""
    return sorted({V // 3, V // 3 + 1, V - 1})


def check(arg, mx, V):
    assert (arg == spoiled(V)[0]).all(), arg.tolist()
    assert mx.isnan().all(), mx.tolist()


# one CTA, clusters of 2, 4 and 8, 64 and 128 columns, pairs; and their ragged ends
@pytest.mark.parametrize("rows, K, N", [(1, 5120, 1024), (1, 5120, 6144), (1, 16, 5), (3, 1024, 301), (33, 2112, 2666), (64, 6144, 256), (100, 3744, 2666),
                                        (128, 512, 384), (130, 1040, 3001), (300, 1152, 700), (2500, 1040, 4999), (1, 640, 40000), (128, 640, 30000)])
def test_products(gpu_lib, rows, K, N):
    g = torch.Generator(device=DEV).manual_seed(rows)
    byte = lambda *s: torch.randint(0, 120, s, device=DEV, dtype=torch.uint8, generator=g)  # noqa: E731
    a, w, sa, sw = byte(rows, K), byte(N, K), torch.rand(rows, -(-K // 128), device=DEV, generator=g), torch.rand(-(-N // 128), -(-K // 128), device=DEV, generator=g)
    w[spoiled(N), K // 2] = 0x7F
    arg, mx = torch.empty(rows, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV)
    tsv.matmul_e4m3_argmax(a, sa, w, sw, arg, maxval=mx)
    check(arg, mx, N)
    if N > 5:  # every product of a row: its first token
        sa[rows // 2, 0] = NAN
        tsv.matmul_e4m3_argmax(a, sa, w, sw, arg, maxval=mx)
        assert arg[rows // 2] == 0 and mx.isnan().all()


@pytest.mark.parametrize("w_dtype", [tsv.F16, tsv.BF16, tsv.Q4_G64, tsv.E4M3_B128])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 14, 40, 64, 200])
@pytest.mark.parametrize("H", [256, 1024])
def test_heads(gpu_lib, rows, H, w_dtype):
    V = 3001
    g = torch.Generator(device=DEV).manual_seed(rows + H)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    scales = biases = None
    if w_dtype == tsv.Q4_G64:
        W = torch.randint(0, 256, (V, H // 2), device=DEV, dtype=torch.uint8, generator=g)
        scales, biases = n(V, H // 64).bfloat16(), n(V, H // 64).bfloat16()
        scales[spoiled(V), H // 128] = NAN
    elif w_dtype == tsv.E4M3_B128:
        W, scales = n(V, H).to(F8).view(torch.uint8), torch.rand(-(-V // 128), -(-H // 128), device=DEV, generator=g)
        W[spoiled(V), H // 2] = 0x7F
    else:
        W = n(V, H).to(torch.float16 if w_dtype == tsv.F16 else torch.bfloat16)
        W[spoiled(V), H // 2] = NAN
    hidden = n(rows, H).bfloat16()
    arg, mx = torch.empty(rows, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV)
    tsv.lm_head_argmax(hidden, W, arg, w_dtype=w_dtype, V=V, scales=scales, biases=biases, maxlogit=mx)
    check(arg, mx, V)
