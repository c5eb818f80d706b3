"""The norm's 8-bit codes: each the nearest one to the value in 64 bits, but where that value lies next to the middle between two codes.

y is off by 2^-17 of itself (tests/test_gpu_rows8.py derives it), its group's scale by as much and half a step, and their quotient in fp32 by two
units in the last place, 2^-22: so a code may be the other neighbour's where the quotient in 64 bits is within 2^-16 + 2^-21 of the middle.
Two calls give the same bits.
"""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv
from oracle import rows8

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows, H", [(2048, 5120), (515, 2573), (64, 12288), (40, 20480), (3000, 256)])
def test_codes(gpu_lib, rows, H, dtype):
    g = torch.Generator(device=DEV).manual_seed(H)
    n = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    loud = 1 + 30 * (torch.rand(H, device=DEV, generator=g) < 0.004)
    x, r, w = (n(rows, H) * loud).to(dtype), (4 * n(rows, H) * loud).to(dtype), (1 + 0.2 * n(H)).to(dtype)

    def run():
        o = torch.empty(rows, H, dtype=torch.uint8, device=DEV), torch.empty(rows, rows8.blocks(H), device=DEV), torch.empty_like(x)
        tsv.add_rms_norm(x, w, eps=1e-6, residual=r, residual_out=o[2], out8=o[0], out8_scale=o[1])
        return o

    one, two = run(), run()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    h = x.double() + r.double()
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    pad = torch.nn.functional.pad(y, (0, rows8.blocks(H) * 128 - H)).view(rows, -1, 128)
    q = (pad / (pad.abs().amax(-1, keepdim=True) / 448)).flatten(1)[:, :H].cpu().numpy()
    near, got = rows8.encode(q), one[0].cpu().numpy()
    a, b = rows8.decode(near), rows8.decode(got)
    i = np.nonzero(a != b)
    # few values lie that near one: of bf16 rows, whose quotients are ratios of short numbers, 215 of 10 million, of fp32 ones 3
    assert len(i[0]) < got.size / 1000
    assert np.all(np.abs(near[i].astype(int) - got[i].astype(int)) == 1)  # neighbours, of one sign
    middle = (a[i] + b[i]) / 2
    assert np.all(np.abs(q[i] - middle) <= np.abs(q[i]) * (2.0 ** -16 + 2.0 ** -21))
