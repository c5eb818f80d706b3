"""The entropy of rows whose logits lie far apart, and of ordinary ones.

entropy = log(sum of exp(z)) + the mean of -z under p, with z = (x - max) / T: z is off by 2^-22 of itself, an exponential by a few steps and
by its z's error, a sum by 2^-15 of itself.  So the entropy is off by (1 + the row's own mean of |z|) 2^-14 at most: a logit without
weight, however far off, has no part in that.
"""
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def rows_of(V, lowest, g):
    x = torch.randn(12, V, generator=g)
    x[0, 1:] = lowest                               # one token left by a mask's lowest value: 0
    x[1] = lowest                                   # all masked alike: log V
    x[2, V // 3] = -lowest * 0.9                    # one logit above everything: 0
    x[3] = lowest
    x[3, [0, V // 2, V - 1]] = torch.tensor([2.0, 2.0, 2.0])  # three alike: log 3
    x[4, 1:] = -INF                                 # 0
    x[5] = -INF
    x[5, [1, V - 1]] = torch.tensor([-3.0, -4.0])
    x[6, V // 2:] = -1e4                            # half of them masked by a finite value
    x[7] = torch.linspace(-30, 30, V)
    x[8] *= 40
    x[9] = 0                                        # log V
    x[10, ::2] = lowest
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [40, 5000, 70001, 248320])
@pytest.mark.parametrize("t", [1.0, 0.6, 1.7])
def test_entropy(gpu_lib, V, t, dtype):
    g = torch.Generator().manual_seed(V)
    x = rows_of(V, torch.finfo(dtype).min, g).clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype).to(DEV)
    x[4, 1:] = x[5, 2:V - 1] = x[5, 0] = -INF
    got = torch.empty(12, device=DEV)
    tsv.token_logprobs(x, entropy=got, temperature=t)
    t32 = float(torch.tensor(t, dtype=torch.float32))
    z = (x.double() - x.double().amax(1, keepdim=True)) / t32
    lp = z - torch.logsumexp(z, 1, keepdim=True)
    p = lp.exp()
    want = torch.special.entr(p).sum(1)
    mean = torch.where(p > 0, p * z.abs(), torch.zeros((), dtype=torch.float64, device=DEV)).sum(1)
    assert (mean < 1e3).all()  # the bound means something in every row
    d = (got.double() - want).abs()
    assert (d <= (1 + mean) * 2.0 ** -14).all(), (d.tolist(), want.tolist())
    assert got[0] == 0 and got[2] == 0 and got[4] == 0
