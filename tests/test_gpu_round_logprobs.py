"""A greedy round gives the same tokens and largest logits whether or not it tells their log probabilities."""
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, T, H, V = 2, 7, 512, 3001
PARENTS = [[-1, 0, 0, 1, 1, 2, 2], [-1, 0, 1, 2, 3, 4, 5]]
SAME = ("argmax", "path", "path_len", "emitted")
INF, NAN = float("inf"), float("nan")


def round_of(w_dtype, logprobs=None, spoil=(), **kw):
    """spoil: (row, feature, value) of the hidden rows."""
    g = torch.Generator().manual_seed(4)
    n = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
    hidden = n(B * T, H)
    for r, c, v in spoil:
        hidden[r, c] = v
    if w_dtype == tsv.E4M3_B128:
        W, ws, wb = n(V, H, dt=torch.float8_e4m3fn), (0.01 + 0.01 * torch.rand(-(-V // 128), H // 128, generator=g)).to(DEV), None
    elif w_dtype == tsv.Q4_G64:
        W = torch.randint(0, 256, (V, H // 2), generator=g, dtype=torch.uint8).to(DEV)
        ws, wb = n(V, H // 64) * 0.01, n(V, H // 64) * 0.01
    else:
        W, ws, wb = n(V, H, dt=torch.bfloat16 if w_dtype == tsv.BF16 else torch.float16), None, None
    return tsv.VerifyRound(T=T, HQ=4, HKV=2, D=64, V=V, kv_dtype=tsv.BF16, w_dtype=w_dtype, max_kv_len=96 + T, hidden=hidden,
                           parents=torch.tensor(PARENTS, dtype=torch.int32, device=DEV),
                           tokens=torch.randint(0, V, (B, T), generator=g, dtype=torch.int32).to(DEV), q=[n(B, T, 4, 64)],
                           k=[n(B, 2, 96 + T, 64)], v=[n(B, 2, 96 + T, 64)], W=W, w_scales=ws, w_biases=wb,
                           kv_len=torch.full((B,), 96 + T, dtype=torch.int32, device=DEV), logprobs=logprobs, **kw)


def bits(t):
    """A NaN counts as one, whatever its bits."""
    return torch.where(t.isnan(), torch.full_like(t, NAN), t).view(torch.int32)


FORMATS = [tsv.F16, tsv.BF16, tsv.Q4_G64, tsv.E4M3_B128]


@pytest.mark.parametrize("w_dtype", FORMATS)
@pytest.mark.parametrize("k", [0, 1, 5])
def test_tokens_and_largest_logits(gpu_lib, w_dtype, k):
    plain, vr = round_of(w_dtype), round_of(w_dtype, k)
    plain.run()
    vr.outs["maxlogit"].fill_(-77)
    vr.run()
    for name in SAME + ("maxlogit",):
        assert torch.equal(vr.outs[name], plain.outs[name]), name
    assert torch.equal(vr.outs["maxlogit"], vr.outs["logits"].amax(1))
    assert torch.equal(vr.outs["argmax"], vr.outs["top_tokens"][:, 0])


@pytest.mark.parametrize("w_dtype", FORMATS)
def test_rows_without_a_distribution(gpu_lib, w_dtype):
    """A NaN or an infinity among a row's features: no log probabilities, and the token that the argmax gives."""
    spoil = ((2, 5, NAN), (4, 9, INF), (11, 300, -INF), (13, 0, NAN))
    plain, vr = round_of(w_dtype, None, spoil), round_of(w_dtype, 5, spoil)
    plain.run()
    vr.run()
    for name in SAME:
        assert torch.equal(vr.outs[name], plain.outs[name]), name
    assert torch.equal(bits(vr.outs["maxlogit"]), bits(plain.outs["maxlogit"]))
    assert (vr.outs["argmax"] >= 0).all() and (vr.outs["argmax"] < V).all()
    assert (vr.outs["top_tokens"][[2, 13]] == -1).all() and vr.outs["logp"][[2, 13]].isnan().all()


def test_captured(gpu_lib):
    plain, vr = round_of(tsv.E4M3_B128), round_of(tsv.E4M3_B128, 3)
    keep = vr.kv_len.clone(), vr.k[0].clone(), vr.v[0].clone()

    def restore(r):
        for to, t in zip((r.kv_len, r.k[0], r.v[0]), keep):
            to.copy_(t)

    vr.run()
    torch.cuda.synchronize()
    vr.capture()
    for seed in (1, 2):
        new = torch.randn(B * T, H, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)
        new[seed] = NAN
        for r in (plain, vr):
            r.hidden.copy_(new)
            restore(r)
        plain.run()
        vr.replay()
        torch.cuda.synchronize()
        for name in SAME:
            assert torch.equal(vr.outs[name], plain.outs[name]), name
        assert torch.equal(bits(vr.outs["maxlogit"]), bits(plain.outs["maxlogit"]))


def test_greedy_tokens(gpu_lib):
    """Rows at any address, rows searched between rows that are not, ties, and values that are no numbers."""
    g = torch.Generator().manual_seed(8)
    for rows, v, k in ((1, 1, 1), (3, 2, 2), (5, 63, 20), (9, 4097, 3), (2000, 301, 2), (2, 248320, 64)):
        x = torch.randn(rows, v, generator=g).to(DEV)
        x[:, v // 3] = 30
        x[:, v // 2] = 30
        want = torch.argmax((x == 30).int(), 1).int()  # the lower of two
        x[1::4, v - 1] = INF
        want[1::4] = v - 1
        x[3::8] = -INF
        want[3::8] = 0
        top, lp = torch.empty(rows, k, dtype=torch.int32, device=DEV), torch.empty(rows, k, device=DEV)
        arg, mx = torch.full((rows,), -7, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV)
        tsv.token_logprobs(x, top_tokens=top, top_logp=lp)
        assert (top[1::4] == -1).all()
        tsv.greedy_tokens(x, top, arg, maxlogit=mx)
        assert torch.equal(arg, want) and torch.equal(mx, x.amax(1))
        arg.fill_(-7)
        tsv.greedy_tokens(x, top, arg)
        assert torch.equal(arg, want)
    x = torch.tensor([[1.0, NAN, 3.0, NAN, INF], [1.0, -NAN, 3.0, 2.0, 3.0]], device=DEV)
    x.view(torch.int32)[0, 1] = x.view(torch.int32)[0, 3] = 0x7FC00000
    x.view(torch.int32)[1, 1] = -0x400000  # a NaN whose sign bit is set
    top = torch.full((2, 1), -1, dtype=torch.int32, device=DEV)
    arg, mx = torch.empty(2, dtype=torch.int32, device=DEV), torch.empty(2, device=DEV)
    tsv.greedy_tokens(x, top, arg, maxlogit=mx)
    assert arg.tolist() == [1, 2] and mx[0].isnan() and mx[1] == 3
