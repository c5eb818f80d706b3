"""The likeliest tokens of rows whose candidates come a few at a time ahead of a stretch where every logit is one.

A part of a row is walked in tiles of 4096 logits, and its list of candidates is looked at between groups of 1, 2, 6, 16, 16 ... tiles.  A
group that brings k / 2 candidates or fewer leaves them in the list as they came; one that brings more than the list holds is read
again.  Every row here has a group of the first kind ahead of one of the second, from every tile on where a part may start.
Tokens are whole decisions: equal to those of a stable sort, largest first.
"""
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TILE = 4096
INF = float("inf")


def spikes(x, tile, n, g, value):
    """n different places of a tile, rising values."""
    at = tile * TILE + torch.randperm(TILE, generator=g)[:n].sort().values.to(x.device)
    x[at] = value + torch.arange(n, device=x.device, dtype=x.dtype)


def rows_of(V, k, starts, g):
    """fp32 rows [n, V]; each kind with its few candidates in the tile after `s`, for every s of starts."""
    ramp = lambda a, b, n: torch.linspace(a, b, n, device=DEV)  # noqa: E731
    few, out = max(1, k // 2), []
    for s in starts:
        c, end = s * TILE, V - (s + 3) * TILE
        for n in {1, few}:
            x = torch.zeros(V, device=DEV)          # a first tile that falls, few peaks, then a raised range
            x[c:c + TILE] = ramp(3, 2, TILE)
            spikes(x, s + 1, n, g, 50)
            x[c + 3 * TILE:] = ramp(10, 11, end)
            out.append(x)
        x = torch.full((V,), -INF, device=DEV)      # a mask that leaves 4 tokens, few likely ones, then everything
        x[c:c + 4] = ramp(1, 2, 4)
        spikes(x, s + 1, min(few, 6), g, 30)
        x[c + 3 * TILE:] = ramp(-3, 3, end)
        out.append(x)
        x = torch.full((V,), -1e4, device=DEV)      # a finite mask, one token, then an open range
        x[(s + 1) * TILE + 77] = 30
        x[c + 3 * TILE:] = torch.randn(end, generator=g).to(DEV)
        out.append(x)
        x = torch.zeros(V, device=DEV)              # flat but for a few peaks, two of them alike, and a raised range at the end
        spikes(x, s + 2, min(few, 2), g, 20)
        x[(s + 1) * TILE + 5] = x[(s + 2) * TILE:(s + 3) * TILE].max()
        x[-3 * TILE:] = 8
        out.append(x)
    return torch.stack(out)


def check(x, k, **kw):
    rows = x.shape[0]
    want = torch.sort(x.float(), dim=1, descending=True, stable=True)
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device=DEV)  # noqa: E731
    o = dict(top_tokens=i32(rows, k), top_logp=torch.empty(rows, k, device=DEV), logp=torch.empty(rows, device=DEV), rank=i32(rows))
    targets = want.indices[:, 0].int()
    tsv.token_logprobs(x, targets, **o, **kw)
    torch.cuda.synchronize()
    wrong = (o["top_tokens"] != want.indices[:, :k]).any(1).nonzero().flatten().tolist()
    assert not wrong, (wrong[:20], o["top_tokens"][wrong[0]].tolist(), want.indices[wrong[0], :k].tolist())
    assert (o["rank"] == 0).all()
    # (x - m) / T off by 2^-22 of itself, a sum of exponentials by 2^-15 of itself
    top = want.values[:, :k].double()
    lp = top - torch.logsumexp(x.double(), 1, keepdim=True)
    fine = torch.isfinite(lp)
    assert torch.equal(fine, torch.isfinite(o["top_logp"]))
    assert ((o["top_logp"].double() - lp).abs() <= lp.abs() * 2.0 ** -21 + 2.0 ** -15)[fine].all()
    assert torch.equal(o["logp"], o["top_logp"][:, 0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k", [2, 5, 20, 64])
def test_one_part(gpu_lib, k, dtype):
    """Rows enough that each is one part: its groups end at the tiles 1, 3, 9 and 25."""
    g = torch.Generator().manual_seed(k)
    x = rows_of(28 * TILE, k, (0, 2, 8), g)
    x = x.repeat(-(-800 // x.shape[0]), 1)
    check(x.to(dtype), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k", [2, 5, 20, 64])
def test_several_parts(gpu_lib, k, dtype):
    """Rows that are split into parts of five tiles and more, which start at any of a row's tiles."""
    g = torch.Generator().manual_seed(k)
    x = rows_of(61 * TILE - 4, k, range(0, 56), g)  # 224 rows and more: three parts or so
    check(x.to(dtype), k)
    check(x[::4].contiguous().to(dtype), k)


def test_unaligned_rows(gpu_lib):
    """Tiles that begin ahead of their row's first logit."""
    g = torch.Generator().manual_seed(7)
    x = rows_of(28 * TILE + 1, 20, (0, 2, 8), g)
    check(x.repeat(-(-800 // x.shape[0]), 1), 20)


@pytest.mark.parametrize("k", [2, 5, 20])
def test_greedy_round_takes_the_same_tokens(gpu_lib, k):
    """One 64-node tree over a vocabulary of 61 tiles: with the likeliest tokens asked for, the walk's tokens stay as they are."""
    T, H, V = 64, 256, 61 * TILE
    g = torch.Generator().manual_seed(k)
    kinds = rows_of(V, 20, range(0, 56, 5), g)[:T].bfloat16().clamp(min=-1e4)
    W = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    W[:, :kinds.shape[0]] = kinds.T
    hidden = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    hidden[torch.arange(T), torch.arange(T) % kinds.shape[0]] = 1
    n = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)  # noqa: E731
    parents = torch.arange(-1, T - 1, dtype=torch.int32, device=DEV)[None]
    best = torch.argmax(kinds.float()[torch.arange(T) % kinds.shape[0]], 1).int()
    tokens = torch.cat([best[:1], best[:-1]])[None].contiguous()  # a chain of the right tokens: all of it is accepted
    q, kv = [n(1, T, 4, 64)], [n(1, 2, 96 + T, 64) for _ in range(2)]

    def ran(**kw):
        vr = tsv.VerifyRound(T=T, HQ=4, HKV=2, D=64, V=V, kv_dtype=tsv.BF16, w_dtype=tsv.BF16, max_kv_len=96 + T, hidden=hidden, parents=parents,
                             tokens=tokens, q=q, k=[kv[0].clone()], v=[kv[1].clone()], W=W,
                             kv_len=torch.full((1,), 96 + T, dtype=torch.int32, device=DEV), **kw)
        vr.run()
        torch.cuda.synchronize()
        return vr

    plain, vr = ran(), ran(logprobs=k)
    assert torch.equal(plain.outs["argmax"], best)
    for name in ("argmax", "path", "path_len", "emitted"):
        assert torch.equal(vr.outs[name], plain.outs[name]), name
    assert torch.equal(vr.kv_len, plain.kv_len)
