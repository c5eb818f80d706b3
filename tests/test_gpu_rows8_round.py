"""A verify round whose last norm, 8-bit LM head and log probabilities run in it, against the calls' oracle."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_array_gb300 as tsv
from oracle import rows8

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, T, H, V, HQ, HKV, D, S = 2, 7, 512, 3001, 4, 2, 64, 96
PARENTS = [[-1, 0, 0, 1, 1, 2, 2], [-1, 0, 1, 2, 3, 4, 5]]


def round_of(seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
    W = (torch.randn(V, H, generator=g) * 8).to(torch.float8_e4m3fn).to(DEV)
    ws = (0.01 + 0.01 * torch.rand(rows8.blocks(V), rows8.blocks(H), generator=g)).to(DEV)
    norm = dict(x=n(B * T, H), weight=(1 + 0.1 * torch.randn(H, generator=g)).bfloat16().to(DEV), eps=1e-6, residual=n(B * T, H),
                residual_out=torch.empty(B * T, H, dtype=torch.bfloat16, device=DEV))
    d = dict(T=T, HQ=HQ, HKV=HKV, D=D, V=V, kv_dtype=tsv.BF16, w_dtype=tsv.E4M3_B128, max_kv_len=S + T, norm=norm, hidden=None,
             parents=torch.tensor(PARENTS, dtype=torch.int32, device=DEV), tokens=torch.randint(0, V, (B, T), generator=g, dtype=torch.int32).to(DEV),
             q=[n(B, T, HQ, D)], k=[n(B, HKV, S + T, D)], v=[n(B, HKV, S + T, D)], W=W, w_scales=ws,
             kv_len=torch.full((B,), S + T, dtype=torch.int32, device=DEV))
    return tsv.VerifyRound(**{**d, **kw})


def logits_of(vr):
    """The oracle's logits from the codes that the norm wrote (the norm itself is checked elsewhere)."""
    o = vr.outs
    byte = lambda t: t.cpu().view(torch.uint8).numpy()  # noqa: E731
    return rows8.matmul(byte(o["hidden8"]), o["hidden8_scale"].cpu().numpy(), byte(vr.W), vr.w_scales.cpu().numpy())


def test_greedy_round(gpu_lib):
    vr = round_of()
    vr.run()
    torch.cuda.synchronize()
    assert int(vr.outs["status"][0]) == 0
    h = vr.norm["x"].float() + vr.norm["residual"].float()
    assert torch.equal(vr.norm["residual_out"], h.bfloat16())
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * vr.norm["weight"].float()
    o = vr.outs
    v = o["hidden8"].float() * o["hidden8_scale"].repeat_interleave(128, 1)
    assert ((v - y).abs() <= torch.maximum(y.abs() * 2.0 ** -4, o["hidden8_scale"].repeat_interleave(128, 1) * 2.0 ** -10) * 1.001).all()
    lg = logits_of(vr)
    arg = o["argmax"].cpu().numpy()
    top = np.sort(lg, 1)
    clear = top[:, -1] - top[:, -2] > 1e-3
    assert clear.sum() > 8 and np.array_equal(arg[clear], np.argmax(lg, 1)[clear])
    assert np.allclose(o["maxlogit"].cpu().numpy(), top[:, -1], rtol=1e-5)
    # the same rows in 16 bits, written first and made 8-bit rows by the head
    wide = round_of(hidden=torch.empty(B * T, H, dtype=torch.bfloat16, device=DEV))
    wide.run()
    assert np.mean(wide.outs["argmax"].cpu().numpy() == arg) > 0.7  # bf16 in between moves codes, and few argmaxes


@pytest.mark.parametrize("k", [0, 1, 5])
def test_greedy_round_with_logprobs(gpu_lib, k):
    plain = round_of()
    plain.run()
    vr = round_of(logprobs=k)
    vr.run()
    o = vr.outs
    assert torch.equal(o["argmax"], plain.outs["argmax"]) and torch.equal(o["path"], plain.outs["path"]) and torch.equal(o["kv_len"] if "kv_len" in o else vr.kv_len, plain.kv_len)
    want = rows8.logprobs(logits_of(vr), o["argmax"].cpu().numpy(), 1.0, max(k, 1))
    # against the oracle's own logits: their fp32 rounding (1e-4 at these sizes) is all that differs
    assert np.allclose(o["logp"].cpu().numpy(), want["logp"], atol=2e-4) and np.allclose(o["entropy"].cpu().numpy(), want["entropy"], atol=2e-3)
    assert np.allclose(o["top_logp"].cpu().numpy(), want["top_logp"], atol=2e-4)


def test_sampled_round_captured(gpu_lib):
    u = torch.rand(B * T, generator=torch.Generator().manual_seed(3)).to(DEV)
    vr, eager = (round_of(sample=(0.8, 20, 0.9), uniforms=u, logprobs=4) for _ in range(2))
    keep = vr.kv_len.clone(), [t.clone() for t in vr.k + vr.v]
    vr.run()
    torch.cuda.synchronize()
    vr.capture()

    def restore():
        vr.kv_len.copy_(keep[0])
        for t, c in zip(vr.k + vr.v, keep[1]):
            t.copy_(c)

    restore()
    vr.replay()
    restore()
    vr.replay()
    eager.run()
    torch.cuda.synchronize()
    for n in ("argmax", "logp", "entropy", "top_tokens", "top_logp", "path", "emitted"):
        assert torch.equal(vr.outs[n], eager.outs[n]), n
    want = rows8.logprobs(vr.outs["logits"].cpu().double().numpy(), vr.outs["argmax"].cpu().numpy(), 1.0, 4)
    assert np.array_equal(vr.outs["top_tokens"].cpu().numpy(), want["top_tokens"])
    assert np.allclose(vr.outs["logp"].cpu().numpy(), want["logp"], atol=1e-4)


def test_greedy_round_with_logprobs_captured(gpu_lib):
    vr, eager = round_of(logprobs=3), round_of(logprobs=3)
    keep = vr.kv_len.clone(), [t.clone() for t in vr.k + vr.v]
    vr.run()
    torch.cuda.synchronize()
    vr.capture()
    vr.norm["x"].copy_(eager.norm["x"].flip(0))
    eager.norm["x"].copy_(vr.norm["x"])
    vr.kv_len.copy_(keep[0])
    for t, c in zip(vr.k + vr.v, keep[1]):
        t.copy_(c)
    vr.replay()
    eager.run()
    torch.cuda.synchronize()
    for n in ("argmax", "logp", "entropy", "top_tokens", "top_logp", "path", "emitted"):
        assert torch.equal(vr.outs[n], eager.outs[n]), n


def test_norm_ahead_of_a_16_bit_head(gpu_lib):
    g = torch.Generator().manual_seed(5)
    W = torch.randn(V, H, generator=g).bfloat16().to(DEV)
    vr = round_of(w_dtype=tsv.BF16, W=W, w_scales=None)
    vr.run()
    h = vr.norm["x"].double() + vr.norm["residual"].double()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * vr.norm["weight"].double()
    assert ((vr.hidden.double() - y).abs() <= y.abs() * (2.0 ** -8 + 2.0 ** -17)).all()
    lg = (vr.hidden.double() @ W.double().T).cpu().numpy()
    assert np.allclose(vr.outs["maxlogit"].cpu().numpy(), lg.max(1), rtol=1e-4)


def test_refusals(gpu_lib):
    with pytest.raises(ValueError, match="hidden"):
        round_of(norm=None)
    with pytest.raises(ValueError, match="B \\* T"):
        round_of(norm=dict(x=torch.zeros(3, H, dtype=torch.bfloat16, device=DEV), weight=torch.zeros(H, dtype=torch.bfloat16, device=DEV), eps=1e-6))
