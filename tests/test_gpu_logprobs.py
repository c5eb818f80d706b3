"""Log probabilities, ranks, entropy and likeliest tokens against the fp64 oracle.

Tokens and ranks are whole decisions on the logits as they are: equal.  Floats: z is off by 2^-22 of itself (a difference, the
reciprocal of T and a product, half an fp32 step each); the exponentials by a few steps and by z's error; a sum of up to 512
numbers in a row in one thread, then over threads, by 2^-15 of itself.  So log probabilities are within 2^-21 |z| + 2^-15 and the
entropy within (1 + its own mean of |z|) 2^-14.
"""
import numpy as np
import pytest
import torch

from oracle import rows8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ask(lib, x, targets=None, t=1.0, k=0, rank=True, entropy=True, **kw):
    rows = x.shape[0]
    f, i = lambda *s: torch.full(s, 7.5, device=DEV), lambda *s: torch.full(s, -9, dtype=torch.int32, device=DEV)  # noqa: E731
    o = {}
    if targets is not None:
        o["logp"] = f(rows)
        if rank:
            o["rank"] = i(rows)
    if entropy:
        o["entropy"] = f(rows)
    if k:
        o["top_tokens"], o["top_logp"] = i(rows, k), f(rows, k)
    lib.token_logprobs(x, targets, temperature=t, **o, **kw)
    torch.cuda.synchronize()
    return {n: v.cpu().numpy() for n, v in o.items()}


def check(got, x, targets=None, t=1.0, k=0):
    x = x.detach().cpu().double().numpy()
    want = rows8.logprobs(x, None if targets is None else targets.cpu().numpy(), t, k)
    t32 = float(np.float32(t))
    with np.errstate(all="ignore"):
        spread = np.abs(np.where(np.isfinite(x), x - np.nanmax(np.where(np.isfinite(x), x, -1e30), axis=1, keepdims=True), 0)).max(1) / t32
    for n, v in got.items():
        if n in ("rank", "top_tokens"):
            assert np.array_equal(v, want[n]), (n, v[:3], want[n][:3])
            continue
        fine = np.isfinite(want[n])
        assert np.array_equal(fine, np.isfinite(v)) and np.array_equal(np.isnan(want[n]), np.isnan(v)), n
        with np.errstate(all="ignore"):
            d = np.abs(v - want[n])
        z = spread[:, None] if v.ndim == 2 else spread
        tol = np.broadcast_to((np.abs(np.where(fine, want[n], 0)) * 2.0 ** -21 + 2.0 ** -15) if n != "entropy" else (1 + z) * 2.0 ** -14, v.shape)
        assert np.all(d[fine] <= tol[fine]), (n, d[fine].max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows, V, k", [(1, 1, 1), (3, 2, 2), (2, 64, 64), (5, 63, 20), (4, 1000, 5), (3, 4097, 64), (2, 16384, 1), (7, 20001, 20), (1, 248320, 64),
                                        (160, 5003, 3), (700, 300, 8), (2, 100003, 0)])
def test_logprobs(gpu_lib, rows, V, k, dtype):
    g = np.random.default_rng(rows + V)
    x = torch.from_numpy((3 * g.standard_normal((rows, V))).astype(np.float32)).to(dtype).to(DEV)
    targets = torch.from_numpy(g.integers(0, V, rows).astype(np.int32)).to(DEV)
    targets[0] = int(x[0].float().argmax())
    for t in (1.0, 0.6):
        check(ask(gpu_lib, x, targets, t, k), x, targets, t, k)


def test_parts(gpu_lib):
    x = torch.randn(6, 9001, device=DEV)
    targets = torch.arange(6, dtype=torch.int32, device=DEV) * 1000
    for kw in (dict(targets=targets, entropy=False), dict(targets=targets, rank=False), dict(), dict(k=5, entropy=False), dict(targets=targets, k=64, entropy=False)):
        got = ask(gpu_lib, x, **kw)
        check(got, x, kw.get("targets"), 1.0, kw.get("k", 0))


@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_masks_ties_and_rows_without_a_distribution(gpu_lib, V):
    g = torch.Generator().manual_seed(V)
    x = torch.randn(14, V, generator=g)
    inf = float("inf")
    x[0] = 0.0                                      # all alike
    x[1, 3:] = -inf                                 # three tokens left
    x[2] = -inf                                     # none
    x[3, V // 2] = float("nan")
    x[4, V - 1] = inf
    x[5] = -inf
    x[5, V - 1] = -3.0                              # one left, at the end
    x[6] = torch.randint(0, 3, (V,), generator=g).float()  # many equal ones
    x[7] = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)  # equal, whatever the sign bit
    x[8] = torch.finfo(torch.float32).min           # a mask's lowest value everywhere: even
    x[9, 1:] = torch.finfo(torch.float32).min
    x[10] = torch.linspace(-5, 5, V)                # ascending
    x[11] = torch.linspace(5, -5, V)
    x[12, V // 3] = 3e38
    x = x.to(DEV)
    targets = torch.tensor([V - 1, 5, 0, 1, 2, V - 1, V // 2, V // 2, 7, 0, 9, V, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    for k in (1, 20, 40):
        check(ask(gpu_lib, x, targets, 1.0, k), x, targets, 1.0, k)
    half = x.clamp(-6e4, 6e4).half()
    check(ask(gpu_lib, half, targets, 1.3, 7), half, targets, 1.3, 7)


def test_every_candidate_in_one_place(gpu_lib):
    """The largest values crowd in one thread's or one part's reach, or come one per part."""
    V = 248320
    x = torch.randn(5, V, device=DEV)
    x[0, 1000:1064] += 50
    x[1, 0:256:4] += 50
    x[2, -64:] += 50
    x[3, :: V // 64] += 50
    x[4, 2000:2000 + 64 * 1024:1024] += 50
    targets = torch.tensor([1001, 4, V - 1, 0, 2001], dtype=torch.int32, device=DEV)
    check(ask(gpu_lib, x, targets, 1.0, 64), x, targets, 1.0, 64)


def test_unaligned_rows_same_bits_twice_and_other_streams(gpu_lib):
    base = torch.randn(4 * 50001 + 3, device=DEV)
    x = base[3:].view(4, 50001)
    targets = torch.tensor([0, 1, 2, 50000], dtype=torch.int32, device=DEV)
    one = ask(gpu_lib, x, targets, 1.0, 20)
    check(one, x, targets, 1.0, 20)
    two = ask(gpu_lib, x, targets, 1.0, 20, stream=torch.cuda.Stream())
    for n in one:
        assert np.array_equal(one[n], two[n]), n
    # at another address the sums are taken in another order: each within its tolerance of the exact value
    three = ask(gpu_lib, x.clone(), targets, 1.0, 20, stream=torch.cuda.Stream())
    check(three, x, targets, 1.0, 20)
    same = ask(gpu_lib, x[:1].expand(300, -1).contiguous(), targets[:1].expand(300).contiguous(), 1.0, 20)
    for n in one:  # another number of rows, another split: within the tolerance, whole values equal
        assert np.allclose(same[n][7], one[n][0], rtol=1e-5, atol=1e-5), n


def test_captured(gpu_lib):
    x = torch.randn(3, 60000, device=DEV)
    targets = torch.tensor([5, 6, 7], dtype=torch.int32, device=DEV)
    o = dict(logp=torch.empty(3, device=DEV), entropy=torch.empty(3, device=DEV), top_tokens=torch.empty(3, 9, dtype=torch.int32, device=DEV),
             top_logp=torch.empty(3, 9, device=DEV), rank=torch.empty(3, dtype=torch.int32, device=DEV))
    ws = torch.empty(max(gpu_lib.token_logprobs_workspace_size(3, 60000, 9), 256), dtype=torch.uint8, device=DEV)
    call = lambda: gpu_lib.token_logprobs(x, targets, workspace=ws, **o)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in range(3):
        x.copy_(torch.randn(3, 60000, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        check({n: v.cpu().numpy() for n, v in o.items()}, x, targets, 1.0, 9)


def test_long_rows_of_many(gpu_lib):
    """2^31 logits and more, looked at in the last rows."""
    x = torch.zeros(9000, 248320, dtype=torch.bfloat16, device=DEV)
    x[-1, 248319], x[-1, 5] = 4, 3
    targets = torch.full((9000,), 248319, dtype=torch.int32, device=DEV)
    got = ask(gpu_lib, x, targets, 1.0, 2)
    last = x[-2:]
    check({n: v[-2:] for n, v in got.items()}, last, targets[-2:], 1.0, 2)
    assert (got["rank"][:-1] == 248319).all() and (got["top_tokens"][:-1] == [0, 1]).all()


@pytest.mark.parametrize("rows, V, k", [(400, 9000, 20), (500, 8200, 64), (130, 12289, 33), (760, 700, 64), (761, 4100, 5)])
def test_rows_that_share_the_gpu_unevenly(gpu_lib, rows, V, k):
    """Parts of one or two tiles, the last of a few logits; the first tile masked but for fewer than k logits in some rows."""
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, V, generator=g)
    x[::3, 3 : min(V, 4096)] = float("-inf")
    x[1::5, : V - 70] = float("-inf")
    x[2::7, 10:50] = 9.0
    targets = torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).to(DEV)
    x = x.to(DEV)
    check(ask(gpu_lib, x, targets, 1.0, k), x, targets, 1.0, k)


@pytest.mark.parametrize("V, k", [(248320, 64), (30000, 64), (9000, 20), (40000, 1)])
def test_parts_are_joined(gpu_lib, V, k):
    """The best of many parts: spread evenly, all in one part, in a few parts whose lists are all better than the others', and few left."""
    g = torch.Generator().manual_seed(V + k)
    x = torch.randn(6, V, generator=g)
    x[0, :4096] += 30                       # one part's
    x[1, : V // 3] += 30                    # a third of the parts'
    x[2] = torch.linspace(-9, 9, V)
    x[3, k + 3 :] = float("-inf")           # hardly more than k left
    x[4] = torch.randint(0, 2, (V,), generator=g).float()
    x[4, V // 2 :] += 5
    targets = torch.randint(0, V, (6,), generator=g, dtype=torch.int32).to(DEV)
    x = x.to(DEV)
    check(ask(gpu_lib, x, targets, 1.0, k), x, targets, 1.0, k)
