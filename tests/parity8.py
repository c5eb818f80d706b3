"""A small greedy verify round with the last norm, an 8-bit LM head and log probabilities, and its check against the fp64 oracle."""
import numpy as np
import torch

import tree_speculative_decoding_array_gb300 as tsv
from oracle import rows8

B, T, H, V, HQ, HKV, D, S = 1, 7, 256, 3001, 4, 2, 64, 96
PARENTS = [[-1, 0, 0, 1, 1, 2, 2]]


def build(device="cuda:0", seed=0, k=3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=g).to(dt).to(device)  # noqa: E731
    return tsv.VerifyRound(
        T=T, HQ=HQ, HKV=HKV, D=D, V=V, kv_dtype=tsv.BF16, w_dtype=tsv.E4M3_B128, max_kv_len=S + T, hidden=None, logprobs=k,
        norm=dict(x=n(B * T, H), residual=n(B * T, H), weight=n(H), eps=1e-6),
        parents=torch.tensor(PARENTS, dtype=torch.int32, device=device),
        tokens=torch.randint(0, V, (B, T), generator=g, dtype=torch.int32).to(device), q=[n(B, T, HQ, D)], k=[n(B, HKV, S + T, D)],
        v=[n(B, HKV, S + T, D)], W=n(V, H, dt=torch.float8_e4m3fn), kv_len=torch.full((B,), S + T, dtype=torch.int32, device=device),
        w_scales=(0.01 + 0.01 * torch.rand(rows8.blocks(V), rows8.blocks(H), generator=g)).to(device))


def check(vr):
    """dict(ok, ...): the codes against the norm in fp64, the logits against the product of these codes, the rest against these logits."""
    f64 = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    byte = lambda t: t.cpu().view(torch.uint8).numpy()  # noqa: E731
    o, norm = vr.outs, vr.norm
    codes, scale = byte(o["hidden8"]), o["hidden8_scale"].cpu().numpy()
    _, y = rows8.add_rms_norm(f64(norm["x"]), f64(norm["weight"]), norm["eps"], f64(norm["residual"]))
    per = np.repeat(scale.astype(np.float64), 128, 1)[:, :H]
    codes_ok = bool(np.all(np.abs(rows8.spread(codes, scale, 1) - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * per) * (1 + 2.0 ** -12)))
    W, ws = byte(vr.W), vr.w_scales.cpu().numpy()
    want, logits = rows8.matmul(codes, scale, W, ws), f64(o["logits"])
    # 128 products are added in fp32 per block, at most a whole step each, then scaled and added over the blocks
    bound = np.abs(rows8.spread(codes, scale, 1)) @ np.abs(rows8.spread(W, ws, 128)).T * (128 * 2.0 ** -23 + (rows8.blocks(H) + 2) * 2.0 ** -24)
    lp = rows8.logprobs(logits, o["argmax"].cpu().numpy(), 1.0, o["top_tokens"].shape[1])
    r = dict(codes_ok=codes_ok, logits_ok=bool(np.all(np.abs(logits - want) <= bound)),
             argmax_exact=bool(np.array_equal(o["argmax"].cpu().numpy(), np.argmax(logits, 1))),
             maxlogit_exact=bool(np.array_equal(f64(o["maxlogit"]), logits.max(1))),
             top_exact=bool(np.array_equal(o["top_tokens"].cpu().numpy(), lp["top_tokens"])),
             logp_max_abs=float(max(np.abs(f64(o["logp"]) - lp["logp"]).max(), np.abs(f64(o["top_logp"]) - lp["top_logp"]).max())),
             entropy_max_abs=float(np.abs(f64(o["entropy"]) - lp["entropy"]).max()), dev_status=o["status"].tolist())
    r["ok"] = all(v for n, v in r.items() if n.endswith(("_ok", "_exact"))) and r["logp_max_abs"] < 1e-4 and r["entropy_max_abs"] < 1e-3 and not any(r["dev_status"])
    return r
