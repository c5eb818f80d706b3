"""GPU parity of 4-bit caches: the attention that reads them, the append that quantises, both gathers, a hybrid round.

Tolerance of the attention against fp64 over the stored values.  The tensor-core kernels take K, V and P as 16-bit
operands (fp16: each within 2^-11 of its value; q is bf16, exact in fp16): a score is within e = 2^-11 sum |q| |k| /
sqrt(D) plus as much for fp32 accumulation and exp, which moves a softmax average of V by at most 2 (2 e) max |v|; P and
V add 2 * 2^-11 max |v|; o is rounded to bf16 once, 2^-8 |o|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import append as oap
from oracle import storage as osd

from .test_gpu_append import rot_error_bound

pytestmark = pytest.mark.gpu
DEV = "cuda"


def random_cache(gen, *shape_D):
    """codes uint8 [..., D/2] and fp16 (scale, bias) [..., D/64, 2] of values about N(0, 1.4)."""
    *shape, D = shape_D
    codes = torch.randint(0, 256, (*shape, D // 2), generator=gen, dtype=torch.uint8)
    sc = (0.15 + 0.3 * torch.rand(*shape, D // 64, generator=gen)).half()
    bi = (-7.5 * sc.float() + 0.2 * torch.randn(sc.shape, generator=gen)).half()
    return codes, torch.stack([sc, bi], dim=-1).contiguous()


def values(codes, pair):
    """fp64 values of 4-bit rows."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
    return q * pair[..., 0].double().repeat_interleave(64, dim=-1) + pair[..., 1].double().repeat_interleave(64, dim=-1)


def random_tree(rng, T):
    return [-1] + [int(rng.integers(0, i)) for i in range(1, T)]


def masks(tsv, trees):
    par = torch.tensor(np.array(trees, dtype=np.int32), device=DEV)
    B, T = par.shape
    anc, depth = torch.zeros(B, T, dtype=torch.int64, device=DEV), torch.zeros(B, T, dtype=torch.int32, device=DEV)
    tsv.tree_mask(par, anc, depth)
    return anc, depth


def ref_attention(q, K, V, parents, S, window=0):
    """fp64: q [T, HQ, D], K/V [HKV, S + T, D] -> (o [T, HQ, D], tolerance of the same shape)."""
    T, HQ, D = q.shape
    HKV = K.shape[0]
    G = HQ // HKV
    ok = torch.zeros(T, S + T, dtype=torch.bool)
    for i in range(T):
        ok[i, :S] = True
        j = i
        while j >= 0:
            ok[i, S + j] = True
            j = parents[j]
        if window:
            ok[i, :max(0, S + i - window + 1)] = False
    o, tol = torch.empty(T, HQ, D, dtype=torch.float64), torch.empty(T, HQ, D, dtype=torch.float64)
    for h in range(HQ):
        k, v = K[h // G], V[h // G]
        s = (q[:, h] @ k.T) / math.sqrt(D)
        e = ((q[:, h].abs() @ k.abs().T) / math.sqrt(D) * ok).amax(-1, keepdim=True) * 2.0 ** -11
        o[:, h] = torch.softmax(s.masked_fill(~ok, -math.inf), -1) @ v
        tol[:, h] = 2.0 ** -8 * o[:, h].abs() + (4 * e + 2.0 ** -10) * v.abs().max()
    return o, tol


def attend(tsv, seed, *, B, T, HQ, HKV, D, S_list, layers=1, splits=0, path=0, window=None, s_cap=None, poison=True):
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    s_cap = s_cap or max(S_list) + T + 3
    trees = [random_tree(rng, T) for _ in range(B)]
    anc, _ = masks(tsv, trees)
    L = [dict(q=torch.randn(B, T, HQ, D, generator=gen).bfloat16(), k=random_cache(gen, B, HKV, s_cap, D),
              v=random_cache(gen, B, HKV, s_cap, D)) for _ in range(layers)]
    dev = [dict(q=x["q"].to(DEV), **{n: [t.to(DEV) for t in x[n]] for n in "kv"}) for x in L]
    if poison:  # rows behind a sequence hold whatever was there: NaN and infinite scales
        for x in dev:
            for b, S in enumerate(S_list):
                for n in "kv":
                    x[n][1][b, :, S + T:, :, 0] = float("nan")
                    x[n][1][b, :, S + T:, :, 1] = float("inf")
    o = [torch.full((B, T, HQ, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(layers)]
    kv_len = torch.tensor([S + T for S in S_list], dtype=torch.int32, device=DEV)
    d = tsv.attn_desc([x["q"] for x in dev], [x["k"][0] for x in dev], [x["v"][0] for x in dev], o, kv_len, anc, T=T, HQ=HQ,
                      HKV=HKV, D=D, kv_dtype=tsv.I4_G64, max_kv_len=max(S_list) + T, k_scale=[x["k"][1] for x in dev],
                      v_scale=[x["v"][1] for x in dev], splits=splits, path=path, window=window)
    ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    tsv.tree_verify_attention(d, ws, dev_status=st)
    torch.cuda.synchronize()
    assert st.tolist()[0] == 0
    for l, x in enumerate(L):
        for b, S in enumerate(S_list):
            want, tol = ref_attention(x["q"][b].double(), values(*(t[b, :, :S + T] for t in x["k"])),
                                      values(*(t[b, :, :S + T] for t in x["v"])), trees[b], S, 0 if window is None else window[l])
            got = o[l][b].double().cpu()
            assert torch.isfinite(got).all(), (l, b)
            assert ((got - want).abs() <= tol).all(), (l, b, ((got - want).abs() / tol).max().item())
            # bf16's rounding alone is within 2^-8 of the norm; the 16-bit operands' errors mix signs
            assert (got - want).norm() <= (2.0 ** -8 + 2.0 ** -9) * want.norm(), (l, b)
    return o


PATHS = {"auto": 0, "cores": 1}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T, HQ, HKV", [(1, 6, 1), (1, 24, 4), (2, 2, 2), (3, 8, 1), (5, 12, 2), (16, 24, 4), (33, 6, 2), (64, 6, 1)])
def test_attention_heads_and_trees(gpu_lib, T, HQ, HKV, D, path):
    attend(gpu_lib, T + D, B=2, T=T, HQ=HQ, HKV=HKV, D=D, S_list=[150, 37], path=PATHS[path])


@pytest.mark.parametrize("S", [0, 1, 15, 16, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("T", [1, 4, 21])
@pytest.mark.parametrize("D", [128, 256])
def test_attention_history_lengths(gpu_lib, D, T, S):
    attend(gpu_lib, S + T, B=1, T=T, HQ=6, HKV=1, D=D, S_list=[S])


@pytest.mark.parametrize("splits", [0, 1, 2, 3, 7, 64])
@pytest.mark.parametrize("T", [1, 2, 16, 64])
def test_attention_splits(gpu_lib, T, splits):
    """Lengths from one key to several tiles a split; sequences whose later splits are empty."""
    attend(gpu_lib, T, B=4, T=T, HQ=12, HKV=2, D=256, S_list=[0, 1, 700, 333], splits=splits, layers=2)


@pytest.mark.parametrize("D, T", [(256, 1), (256, 3), (256, 24), (128, 1), (128, 10)])
def test_attention_sliding_window(gpu_lib, D, T):
    attend(gpu_lib, T, B=2, T=T, HQ=8, HKV=2, D=D, S_list=[500, 90], layers=4, window=[0, 1, 64, 200])


@pytest.mark.parametrize("path", [3, 4])
@pytest.mark.parametrize("T, HQ, S_list", [(1, 4, [64]), (3, 24, [300, 5]), (16, 24, [777, 200]), (64, 12, [129, 1000])])
def test_attention_tensor_core_tiles(gpu_lib, T, HQ, S_list, path):
    attend(gpu_lib, T, B=len(S_list), T=T, HQ=HQ, HKV=2, D=256, S_list=S_list, path=path)


def test_attention_wide_scales(gpu_lib):
    """Groups whose scale is 0 (one value), tiny (fp16 subnormal) or large beside ordinary ones."""
    for T in (1, 20):
        gen = torch.Generator().manual_seed(T)
        B, HQ, HKV, D, S = 1, 6, 1, 256, 300
        (kc, kp), (vc, vp) = random_cache(gen, B, HKV, S + T, D), random_cache(gen, B, HKV, S + T, D)
        kp[:, :, ::3, 1, 0], kp[:, :, ::5, 2, 0] = 0.0, 2.0 ** -20
        vp[:, :, ::2, 0, 0], vp[:, :, ::7, 3, 0], vp[:, :, ::4, 2] = 0.0, 2.0 ** -22, torch.tensor([40.0, -300.0]).half()
        q = torch.randn(B, T, HQ, D, generator=gen).bfloat16()
        par = [random_tree(np.random.default_rng(T), T)]
        anc, _ = masks(gpu_lib, par)
        o = torch.empty(B, T, HQ, D, dtype=torch.bfloat16, device=DEV)
        dv = [t.to(DEV) for t in (q, kc, kp, vc, vp)]
        d = gpu_lib.attn_desc([dv[0]], [dv[1]], [dv[3]], [o], torch.tensor([S + T], dtype=torch.int32, device=DEV), anc, T=T,
                              HQ=HQ, HKV=HKV, D=D, kv_dtype=gpu_lib.I4_G64, max_kv_len=S + T, k_scale=[dv[2]], v_scale=[dv[4]])
        ws = torch.empty(max(gpu_lib.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
        gpu_lib.tree_verify_attention(d, ws)
        want, tol = ref_attention(q[0].double(), values(kc[0], kp[0]), values(vc[0], vp[0]), par[0], S)
        # a group's error is its own: the tolerance per 64 features takes that group's largest |v|
        vmax = values(vc[0], vp[0]).abs()[0].view(-1, 4, 64).amax(dim=(0, 2)).repeat_interleave(64)
        got = o[0].double().cpu()
        small = (tol - 2.0 ** -8 * want.abs()) / values(vc[0], vp[0]).abs().max()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + small * vmax).all()


@pytest.mark.parametrize("T, path", [(1, 0), (2, 0), (16, 0), (4, 1)])
def test_attention_nan_in_a_row_that_is_masked_everywhere_else(gpu_lib, T, path):
    """A sequence's bad length is reported and left; the others are computed."""
    gen = torch.Generator().manual_seed(1)
    B, HQ, HKV, D, S = 3, 6, 1, 256, 100
    k, v = ([t.to(DEV) for t in random_cache(gen, B, HKV, S + T, D)] for _ in "kv")
    q = torch.randn(B, T, HQ, D, generator=gen).bfloat16().to(DEV)
    anc, _ = masks(gpu_lib, [[-1] + list(range(T - 1))] * B)
    for bad in (T - 1, S + T + 1, -5, 1 << 30):
        o = torch.full((B, T, HQ, D), 7.0, dtype=torch.bfloat16, device=DEV)
        kv_len = torch.tensor([S + T, bad, S + T], dtype=torch.int32, device=DEV)
        d = gpu_lib.attn_desc([q], [k[0]], [v[0]], [o], kv_len, anc, T=T, HQ=HQ, HKV=HKV, D=D, kv_dtype=gpu_lib.I4_G64,
                              max_kv_len=S + T, k_scale=[k[1]], v_scale=[v[1]], path=path)
        ws = torch.empty(max(gpu_lib.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
        st = torch.zeros(4, dtype=torch.int32, device=DEV)
        gpu_lib.tree_verify_attention(d, ws, dev_status=st)
        torch.cuda.synchronize()
        assert st.tolist()[:2] == [gpu_lib.DEV_BAD_KV_LEN, 1]
        assert (o[1] == 7.0).all() and not (o[0] == 7.0).all() and torch.isfinite(o).all()


# ----------------------------------------------------------------------------- append
@pytest.mark.parametrize("D, rot_dim, interleaved", [(64, 64, False), (128, 32, False), (256, 256, False), (256, 64, True), (64, 2, True)])
@pytest.mark.parametrize("T", [1, 7, 64])
def test_append_quantises(gpu_lib, T, D, rot_dim, interleaved):
    rng = np.random.default_rng(T + D)
    B, HQ, HKV, layers, S_list, base = 2, 4, 2, 2, [0, 77], 1e4
    s_cap = max(S_list) + T + 4
    trees = [random_tree(rng, T) for _ in range(B)]
    anc, depth = masks(gpu_lib, trees)
    bf = lambda *s, m=1.0: (torch.from_numpy(rng.standard_normal(s)) * m).bfloat16().to(DEV)  # noqa: E731
    x = [dict(q=bf(B, T, HQ, D), kn=bf(B, T, HKV, D, m=2.0), vn=bf(B, T, HKV, D)) for _ in range(layers)]
    for y in x:
        y["vn"][0, 0, 0] = 1.5  # one value: scale 0, codes 0
        y["qo"] = torch.empty_like(y["q"])
        for n in "kv":
            y[n] = torch.full((B, HKV, s_cap, D // 2), 0xA5, dtype=torch.uint8, device=DEV)
            y[n + "s"] = torch.full((B, HKV, s_cap, D // 64, 2), 0.25, dtype=torch.float16, device=DEV)
    g = lambda n: [y[n] for y in x]  # noqa: E731
    d = gpu_lib.append_desc(g("q"), g("qo"), g("kn"), g("vn"), g("k"), g("v"), depth, T=T, HQ=HQ, HKV=HKV, D=D,
                            kv_dtype=gpu_lib.I4_G64, rot_dim=rot_dim, rope_base=base, interleaved=interleaved,
                            k_scale=g("ks"), v_scale=g("vs"))
    kv_len = torch.tensor(S_list, dtype=torch.int32, device=DEV)
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    gpu_lib.tree_append(d, kv_len, dev_status=st)
    torch.cuda.synchronize()
    assert st.tolist()[0] == 0 and kv_len.tolist() == [S + T for S in S_list]
    for y in x:
        kn, vn = y["kn"].double().cpu().numpy(), y["vn"].double().cpu().numpy()
        bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        for b, S in enumerate(S_list):
            outside = [c for c in range(s_cap) if not S <= c < S + T]
            for n in "kv":
                assert (y[n][b][:, outside] == 0xA5).all() and (y[n + "s"][b][:, outside] == 0.25).all()
            pos = oap.node_positions(trees[b], S)
            for i in range(T):
                for h in range(HKV):
                    codes, pair = oap.quantize_token4(vn[b, i, h])
                    got = y["v"][b, h, S + i].cpu().numpy()
                    assert np.array_equal(osd.unpack_q4(got[None])[0], codes)
                    assert np.array_equal(bits(y["vs"][b, h, S + i]), pair)
                    # K: the rotation's fp32 error moves an extreme, and with it scale and bias, by at most delta
                    want = oap.rope(kn[b, i, h], pos[i], base, rot_dim, interleaved)
                    delta = rot_error_bound(kn[b, i, h], rot_dim, interleaved).max()
                    w = want.reshape(-1, 64)
                    sc, bi = (osd.f16(bits(y["ks"][b, h, S + i]))[:, c] for c in (0, 1))
                    for val, exact, dd in ((sc, (w.max(1) - w.min(1)) / 15, 2 * delta / 15), (bi, w.min(1), delta)):
                        # fp16 rounding is within 2^-11 of the value; fp32 steps within 2^-23
                        assert np.all(np.abs(val - exact) <= (2.0 ** -11 + 2.0 ** -22) * np.abs(exact) + dd + 2.0 ** -24)
                    y4 = osd.kv_values(4, y["k"][b, h, S + i].cpu().numpy(), bits(y["ks"][b, h, S + i]))
                    step = np.repeat(sc, 64)
                    edge = 15 * step * 2.0 ** -10 + np.repeat(np.abs(w).max(1), 64) * 2.0 ** -10
                    assert np.all(np.abs(y4 - want) <= step / 2 + edge + 2 * delta)


# ----------------------------------------------------------------------------- gathers
@pytest.mark.parametrize("D", [64, 128, 256])
def test_gathers_move_rows_with_their_pairs(gpu_lib, D):
    gen = torch.Generator().manual_seed(D)
    B, HKV, S, T, layers = 3, 2, 40, 9, 2
    s_cap = S + T + 2
    x = [{n: [t.to(DEV) for t in random_cache(gen, B, HKV, s_cap, D)] for n in "kv"} for _ in range(layers)]
    old = [{n: [t.clone() for t in y[n]] for n in "kv"} for y in x]
    g = lambda n, i: [y[n][i] for y in x]  # noqa: E731
    d = gpu_lib.kv_desc(g("k", 0), g("v", 0), HKV=HKV, D=D, kv_dtype=gpu_lib.I4_G64, k_scale=g("k", 1), v_scale=g("v", 1))
    paths = [[0, 3, 4, 8], [0, 1, 2], list(range(T))]
    kv_len = torch.full((B,), S + T, dtype=torch.int32, device=DEV)
    path = torch.tensor([p + [-1] * (T - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    plen = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV)
    gpu_lib.kv_gather_positions(d, kv_len, path, plen, T)
    assert kv_len.tolist() == [S + len(p) for p in paths]
    for y, z in zip(x, old):
        for n in "kv":
            for i in (0, 1):
                for b, p in enumerate(paths):
                    want = z[n][i][b].clone()
                    want[:, S:S + len(p)] = z[n][i][b][:, [S + j for j in p]]
                    assert torch.equal(y[n][i][b], want)
    # the absolute form, over several chunks of rows
    kept = [sorted(np.random.default_rng(b).choice(S + T, size=n, replace=False).tolist()) for b, n in enumerate((30, 0, 47))]
    for y, z in zip(x, old):
        for n in "kv":
            for i in (0, 1):
                y[n][i].copy_(z[n][i])
    kv_len.fill_(S + T)
    gpu_lib.gather_positions(d, kv_len, torch.tensor([k + [0] * (47 - len(k)) for k in kept], dtype=torch.int32, device=DEV),
                             torch.tensor([len(k) for k in kept], dtype=torch.int32, device=DEV))
    assert kv_len.tolist() == [len(k) for k in kept]
    for y, z in zip(x, old):
        for n in "kv":
            for i in (0, 1):
                for b, k in enumerate(kept):
                    want = z[n][i][b].clone()
                    want[:, :len(k)] = z[n][i][b][:, k]
                    assert torch.equal(y[n][i][b], want)


def test_a_long_absolute_gather(gpu_lib):
    gen = torch.Generator().manual_seed(2)
    B, HKV, D, n = 1, 1, 64, 3000
    k, v = ([t.to(DEV) for t in random_cache(gen, B, HKV, n, D)] for _ in "kv")
    old = [t.clone() for t in k + v]
    kept = sorted(np.random.default_rng(0).choice(n, size=2100, replace=False).tolist())
    d = gpu_lib.kv_desc([k[0]], [v[0]], HKV=HKV, D=D, kv_dtype=gpu_lib.I4_G64, k_scale=[k[1]], v_scale=[v[1]])
    kv_len = torch.tensor([n], dtype=torch.int32, device=DEV)
    gpu_lib.gather_positions(d, kv_len, torch.tensor([kept], dtype=torch.int32, device=DEV),
                             torch.tensor([len(kept)], dtype=torch.int32, device=DEV))
    for got, was in zip(k + v, old):
        assert torch.equal(got[:, :, :len(kept)], was[:, :, kept]) and torch.equal(got[:, :, len(kept):], was[:, :, len(kept):])


# ----------------------------------------------------------------------------- a hybrid target's round
@pytest.mark.parametrize("captured", [False, True])
def test_hybrid_round(gpu_lib, captured):
    """Two rounds of a hybrid target (4-bit caches, recurrent layers) through VerifyRound: append, attention, recurrent
    layers, head, walk, gather and commit, each round's state feeding the next."""
    tsv = gpu_lib
    B, T, HQ, HKV, D, H, V, L, R, HK, HV = 2, 6, 12, 2, 256, 512, 2048, 2, 2, 2, 4
    S0, cap = [70, 33], 128
    gen, rng = torch.Generator().manual_seed(5), np.random.default_rng(5)
    r = lambda *s, m=1.0: (torch.randn(*s, generator=gen) * m).to(DEV)  # noqa: E731
    caches = [{n: [t.to(DEV) for t in random_cache(gen, B, HKV, cap, D)] for n in "kv"} for _ in range(L)]
    c = lambda n, i: [y[n][i] for y in caches]  # noqa: E731
    bf = lambda *s, m=1.0: r(*s, m=m).bfloat16()  # noqa: E731
    gdn = dict(q=[bf(B, T, HK, 128) for _ in range(R)], k=[bf(B, T, HK, 128) for _ in range(R)],
               v=[bf(B, T, HV, 128) for _ in range(R)], g=[-r(B, T, HV).abs() for _ in range(R)],
               beta=[torch.sigmoid(r(B, T, HV)) for _ in range(R)], state=[r(B, HV, 128, 128, m=0.3) for _ in range(R)])
    vr = tsv.VerifyRound(T=T, HQ=HQ, HKV=HKV, D=D, V=V, kv_dtype=tsv.I4_G64, w_dtype=tsv.BF16, max_kv_len=cap,
                         parents=torch.zeros(B, T, dtype=torch.int32, device=DEV), tokens=torch.zeros(B, T, dtype=torch.int32, device=DEV),
                         q=[bf(B, T, HQ, D) for _ in range(L)], k=c("k", 0), v=c("v", 0), hidden=bf(B * T, H), W=bf(V, H, m=0.05),
                         kv_len=torch.tensor(S0, dtype=torch.int32, device=DEV), k_scale=c("k", 1), v_scale=c("v", 1),
                         q_in=[bf(B, T, HQ, D) for _ in range(L)], k_new=[bf(B, T, HKV, D) for _ in range(L)],
                         v_new=[bf(B, T, HKV, D) for _ in range(L)], rot_dim=64, rope_base=1e4, gdn=gdn)
    par0 = [[-1, 0, 0, 1, 1, 4], [-1, 0, 1, 1, 3, 0]]
    vr.parents.copy_(torch.tensor(par0, dtype=torch.int32))
    logits = vr.hidden.double() @ vr.W.double().T
    am = logits.argmax(-1).view(B, T).cpu().numpy()
    plan = [[0, 1, 4], [0]]  # accepted paths: make the drafted tokens match the head's choices along them
    tok = rng.integers(0, V, (B, T))
    tok[tok == am[0, 0]] += 1
    for b, p in enumerate(plan):
        tok[b, 1:] = -1 - np.arange(T - 1)
        for a, n in zip(p, p[1:]):
            tok[b, n] = am[b, a]
    vr.tokens.copy_(torch.tensor(tok, dtype=torch.int32))
    lens, states = list(S0), [s.clone() for s in gdn["state"]]
    start = [[t.clone() for n in "kv" for t in y[n]] for y in caches]
    if captured:
        keep = vr.kv_len.clone()
        vr.run()  # warm the lazily loaded kernels, then put everything back
        torch.cuda.synchronize()
        vr.kv_len.copy_(keep)
        for s, t in zip(gdn["state"], states):
            s.copy_(t)
        for y, z in zip(caches, start):
            for t, u in zip([t for n in "kv" for t in y[n]], z):
                t.copy_(u)
        vr.capture()
    for _ in range(2):
        out = vr.replay() if captured else vr.run()
        torch.cuda.synchronize()
        assert out["status"].tolist()[0] == 0
        assert [out["path"][b, :out["path_len"][b]].tolist() for b in range(B)] == plan
        for l in range(R):
            for b in range(B):
                one = lambda n: gdn[n][l][b].double().cpu().numpy()  # noqa: E731
                from oracle import gdn as og
                st = states[l][b].double().cpu().numpy()
                want = og.tree_verify(one("q"), one("k"), one("v"), one("g"), one("beta"), st, par0[b])
                got = out["gdn_o"][l][b].double().cpu().numpy()
                assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10)
                new = og.commit(one("q"), one("k"), one("v"), one("g"), one("beta"), st, plan[b])
                assert np.abs(gdn["state"][l][b].double().cpu().numpy() - new).max() <= 2.0 ** -17
        for l in range(L):
            for b in range(B):
                n, S = lens[b], lens[b]
                # the cache's accepted rows were moved behind the history; attention read them at their block slots,
                # so the reference rebuilds the block from the inputs
                K, Vv = (np.zeros((HKV, S + T, D)) for _ in "kv")
                for x, name, X in ((vr.k_new, "k", K), (vr.v_new, "v", Vv)):
                    codes, pair = caches[l][name]
                    X[:, :S] = values(codes[b, :, :S].cpu(), pair[b, :, :S].cpu()).numpy()
                    pos = oap.node_positions(par0[b], S)
                    for i in range(T):
                        for h in range(HKV):
                            row = x[l][b, i, h].double().cpu().numpy()
                            row = oap.rope(row, pos[i], 1e4, 64) if name == "k" else row
                            cd, pr = oap.quantize_token4(row)
                            X[h, S + i] = osd.kv_values(4, (cd[0::2] | (cd[1::2] << 4)).astype(np.uint8), pr)
                want, tol = ref_attention(vr.q[l][b].double().cpu(), torch.from_numpy(K), torch.from_numpy(Vv), par0[b], S)
                # a block key on a rounding boundary may take the code beside the oracle's: one step of a K value
                got = out["o"][l][b].double().cpu()
                assert ((got - want).abs() <= tol + 0.05).all()
                for j, i in enumerate(plan[b]):
                    codes, pair = caches[l]["v"]
                    got_row = values(codes[b, :, S + j].cpu(), pair[b, :, S + j].cpu()).numpy()
                    assert np.array_equal(got_row, Vv[:, S + i])
        lens = [n + len(p) for n, p in zip(lens, plan)]
        assert vr.kv_len.tolist() == lens
        states = [s.clone() for s in gdn["state"]]


def test_rows_that_are_not_finite_stay_with_the_nodes_that_see_them(gpu_lib):
    """A branch whose K and V rows hold NaN, infinities or values beyond fp16 is appended to the 4-bit cache; every node
    that does not attend to it computes what it computes without it."""
    tsv, T, HQ, HKV, D, S = gpu_lib, 7, 6, 1, 256, 90
    par = [-1, 0, 0, 1, 2, 4, 3]  # node 2 and its descendants 4, 5 are the bad branch
    anc, depth = masks(tsv, [par])
    for head_rows in (1, 6):  # few query rows and many
        out = []
        for bad in (False, True):
            gen = torch.Generator().manual_seed(3)
            kc, vc = ([t.to(DEV) for t in random_cache(gen, 1, HKV, S + T, D)] for _ in "kv")
            q, kn, vn = (torch.randn(1, T, n, D, generator=gen).bfloat16().to(DEV) for n in (head_rows, HKV, HKV))
            if bad:
                for x in (kn, vn):
                    x[0, 2], x[0, 4, 0, ::3], x[0, 5, 0, ::2] = float("nan"), float("inf"), 1e30
            o, qo = torch.empty_like(q), torch.empty_like(q)
            d = tsv.append_desc([q], [qo], [kn], [vn], [kc[0]], [vc[0]], depth, T=T, HQ=head_rows, HKV=HKV, D=D, kv_dtype=tsv.I4_G64,
                                rot_dim=64, rope_base=1e4, k_scale=[kc[1]], v_scale=[vc[1]])
            kv_len = torch.tensor([S], dtype=torch.int32, device=DEV)
            tsv.tree_append(d, kv_len)
            assert torch.isfinite(kc[1]).all() and torch.isfinite(vc[1]).all()
            assert values(vc[0], vc[1]).abs().max() < 65520
            a = tsv.attn_desc([qo], [kc[0]], [vc[0]], [o], kv_len, anc, T=T, HQ=head_rows, HKV=HKV, D=D, kv_dtype=tsv.I4_G64,
                              max_kv_len=S + T, k_scale=[kc[1]], v_scale=[vc[1]])
            ws = torch.empty(max(tsv.attention_workspace_size(a), 16), dtype=torch.uint8, device=DEV)
            tsv.tree_verify_attention(a, ws)
            torch.cuda.synchronize()
            out.append(o.clone())
        clear = [0, 1, 3, 6]
        assert torch.equal(out[0][0, clear], out[1][0, clear])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_of_rows_that_are_not_finite(gpu_lib, D):
    """The stored form of NaN, infinities and values beyond fp16, as the oracle's (V rows are not rotated)."""
    tsv, rows = gpu_lib, []
    for what in range(7):
        x = torch.randn(D, generator=torch.Generator().manual_seed(what))
        if what == 0:
            x[:] = float("nan")
        elif what == 1:
            x[::3] = float("nan")
        elif what == 2:
            x[5], x[6] = float("inf"), -float("inf")
        elif what == 3:
            x[:] = float("inf")
        elif what == 4:
            x[:] = 1e30
            x[::2] = -3e4
        elif what == 5:
            x[:64] = -float("inf")
        rows.append(x)
    T = len(rows)
    vn = torch.stack(rows)[None, :, None].bfloat16().to(DEV)
    kc, vc = ([torch.zeros(1, 1, T, D // 2, dtype=torch.uint8, device=DEV), torch.zeros(1, 1, T, D // 64, 2, dtype=torch.float16, device=DEV)]
              for _ in "kv")
    q = torch.zeros(1, T, 1, D, dtype=torch.bfloat16, device=DEV)
    d = tsv.append_desc([q], [torch.empty_like(q)], [torch.zeros_like(vn)], [vn], [kc[0]], [vc[0]], torch.zeros(1, T, dtype=torch.int32, device=DEV),
                        T=T, HQ=1, HKV=1, D=D, kv_dtype=tsv.I4_G64, rot_dim=32, rope_base=1e4, k_scale=[kc[1]], v_scale=[vc[1]])
    tsv.tree_append(d, torch.zeros(1, dtype=torch.int32, device=DEV))
    for i in range(T):
        codes, pair = oap.quantize_token4(vn[0, i, 0].double().cpu().numpy())
        got = vc[0][0, 0, i].cpu().numpy()
        assert (np.stack([got & 15, got >> 4], -1).reshape(-1) == codes).all(), i
        assert (vc[1][0, 0, i].cpu().numpy().view(np.uint16) == pair).all(), i


@pytest.mark.parametrize("T", [1, 20])
def test_offsets_beyond_32_bits(gpu_lib, T):
    """The second sequence of a cache whose buffers pass 2^31 bytes and 2^32 codes."""
    tsv, HQ, HKV, D, S = gpu_lib, 6, 1, 256, 500
    cap = (1 << 31) // (D // 2) + 1000
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(2, T, HQ, D, generator=gen).bfloat16()
    parts = [[random_cache(gen, HKV, S + T, D) for _ in "kv"] for _ in range(2)]
    k, v = (torch.empty(2, HKV, cap, D // 2, dtype=torch.uint8, device=DEV) for _ in "kv")
    ks, vs = (torch.empty(2, HKV, cap, D // 64, 2, dtype=torch.float16, device=DEV) for _ in "kv")
    for b in range(2):
        for (codes, pair), c, s in zip(parts[b], (k, v), (ks, vs)):
            c[b, :, :S + T], s[b, :, :S + T] = codes.to(DEV), pair.to(DEV)
    par = [random_tree(np.random.default_rng(T), T) for _ in range(2)]
    anc, _ = masks(tsv, par)
    o = torch.empty(2, T, HQ, D, dtype=torch.bfloat16, device=DEV)
    kv_len = torch.full((2,), S + T, dtype=torch.int32, device=DEV)
    d = tsv.attn_desc([q.to(DEV)], [k], [v], [o], kv_len, anc, T=T, HQ=HQ, HKV=HKV, D=D, kv_dtype=tsv.I4_G64, max_kv_len=S + T,
                      k_scale=[ks], v_scale=[vs])
    ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
    tsv.tree_verify_attention(d, ws)
    for b in range(2):
        want, tol = ref_attention(q[b].double(), *(values(*x) for x in parts[b]), par[b], S)
        assert ((o[b].double().cpu() - want).abs() <= tol).all()
    # and the gather of the block behind it
    if T > 1:
        path = torch.tensor([[0, 2, 5] + [-1] * (T - 3)] * 2, dtype=torch.int32, device=DEV)
        tsv.kv_gather_positions(tsv.kv_desc([k], [v], HKV=HKV, D=D, kv_dtype=tsv.I4_G64, k_scale=[ks], v_scale=[vs]), kv_len, path,
                                torch.full((2,), 3, dtype=torch.int32, device=DEV), T)
        for (codes, pair), c, s in zip(parts[1], (k, v), (ks, vs)):
            assert torch.equal(c[1, :, S + 2].cpu(), codes[:, S + 5]) and torch.equal(s[1, :, S + 1].cpu(), pair[:, S + 2])


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("at", [0, 9000])
@pytest.mark.parametrize("T, D", [(1, 256), (2, 256), (20, 256), (1, 128), (3, 64)])
def test_small_values_behind_a_key_that_draws_most_of_the_weight(gpu_lib, T, D, at, big):
    """16000 keys of values up to 15 * 2^-9, each e^-11 behind one key whose values are 0: together a fifth of the
    weight.  With `big`, values of one late key reach 15 * 100."""
    tsv, HQ, S = gpu_lib, 6, 16000
    gen = torch.Generator().manual_seed(T)
    pair = lambda s, b: torch.tensor([s, b]).half()  # noqa: E731
    k, v = ([torch.zeros(1, S + T, D // 2, dtype=torch.uint8), torch.zeros(1, S + T, D // 64, 2, dtype=torch.float16)] for _ in "kv")
    k[1][0, at] = pair(0.0, 11.0 / D ** 0.5)
    v[0][:] = torch.randint(0, 256, v[0].shape, generator=gen)
    v[1][:] = pair(2.0 ** -9, 0.0)
    v[1][0, at] = 0.0
    if big:
        v[1][0, S - 10] = pair(100.0, 0.0)
    q = torch.ones(1, T, HQ, D).bfloat16()
    par = [list(range(-1, T - 1))]
    anc, _ = masks(tsv, par)
    o = torch.empty(1, T, HQ, D, dtype=torch.bfloat16, device=DEV)
    dev = [[x[None].to(DEV) for x in y] for y in (k, v)]
    d = tsv.attn_desc([q.to(DEV)], [dev[0][0]], [dev[1][0]], [o], torch.tensor([S + T], dtype=torch.int32, device=DEV), anc, T=T, HQ=HQ,
                      HKV=1, D=D, kv_dtype=tsv.I4_G64, max_kv_len=S + T, k_scale=[dev[0][1]], v_scale=[dev[1][1]], splits=1)
    ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
    tsv.tree_verify_attention(d, ws)
    want, _ = ref_attention(q[0].double(), values(*k), values(*v), par[0], S)
    # P (times a scale) in fp16 is off by 2^-11 of itself and 2^-25 absolutely, relative to the largest P of 1 / 4 or more
    # (one of 2^-8 on the tiles of 128 rows): 16000 such keys add up to 2^-9 of the weight.  The bias sum is zero here.
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 16000 * 2.0 ** -25 * 4) * 15 * 2.0 ** -9 + (2.0 ** -9 * want.abs() if big else 0)
    assert ((o[0].double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("T, HQ, HKV, D, path", [(1, 6, 1, 256, 0), (5, 4, 2, 256, 0), (16, 24, 4, 256, 0), (1, 8, 2, 128, 0), (20, 6, 1, 64, 0),
                                                 (4, 6, 2, 128, 0)])
def test_a_query_row_that_is_not_finite(gpu_lib, T, HQ, HKV, D, path, splits):
    """NaN in one row of q (all of it, or one feature), infinities and values beyond fp16: NaN comes out of that row (zeros
    would hide a broken model), the other rows are bit for bit as without it."""
    tsv, B, S = gpu_lib, 2, 300
    gen = torch.Generator().manual_seed(T + D)
    k, v = ([t.to(DEV) for t in random_cache(gen, B, HKV, S + T, D)] for _ in "kv")
    anc, _ = masks(tsv, [random_tree(np.random.default_rng(b), T) for b in range(B)])
    clean = torch.randn(B, T, HQ, D, generator=gen).bfloat16().to(DEV)
    kv_len = torch.tensor([S + T, S + T - 100], dtype=torch.int32, device=DEV)

    def run(q):
        o = torch.full((B, T, HQ, D), 7.0, dtype=torch.bfloat16, device=DEV)
        d = tsv.attn_desc([q], [k[0]], [v[0]], [o], kv_len, anc, T=T, HQ=HQ, HKV=HKV, D=D, kv_dtype=tsv.I4_G64, max_kv_len=S + T,
                          k_scale=[k[1]], v_scale=[v[1]], splits=splits, path=path)
        ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
        tsv.tree_verify_attention(d, ws)
        torch.cuda.synchronize()
        return o

    want = run(clean)
    b, i, h = 1, T // 2, HQ - 1
    for bad in (float("nan"), "one nan", float("inf"), -float("inf"), 1e30):
        q = clean.clone()
        if bad == "one nan":
            q[b, i, h, 5] = float("nan")
        else:
            q[b, i, h] = bad
        o = run(q)
        assert torch.isnan(o[b, i, h]).all(), bad
        o[b, i, h] = want[b, i, h]
        assert torch.equal(o, want), bad


@pytest.mark.parametrize("T, HQ", [(7, 1), (7, 6)])
def test_a_nan_in_a_row_that_is_masked(gpu_lib, T, HQ):
    """Pairs of rows behind kv_len may be NaN; q rows of another sequence may be; neither reaches a row that does not see
    them, in the kernels of few and of many query rows."""
    tsv, HKV, D, S, B = gpu_lib, 1, 256, 90, 2
    gen = torch.Generator().manual_seed(T)
    k, v = ([t.to(DEV) for t in random_cache(gen, B, HKV, S + T + 40, D)] for _ in "kv")
    anc, _ = masks(tsv, [[-1, 0, 0, 1, 2, 4, 3]] * B)
    q = torch.randn(B, T, HQ, D, generator=gen).bfloat16().to(DEV)
    outs = []
    for bad in (False, True):
        if bad:
            q[1] = float("nan")
            for x in (k, v):
                x[1][:, :, S + T:] = float("nan")
        o = torch.empty(B, T, HQ, D, dtype=torch.bfloat16, device=DEV)
        d = tsv.attn_desc([q], [k[0]], [v[0]], [o], torch.full((B,), S + T, dtype=torch.int32, device=DEV), anc, T=T, HQ=HQ, HKV=HKV, D=D,
                          kv_dtype=tsv.I4_G64, max_kv_len=S + T, k_scale=[k[1]], v_scale=[v[1]])
        ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
        tsv.tree_verify_attention(d, ws)
        torch.cuda.synchronize()
        outs.append(o.clone())
    assert torch.equal(outs[0][0], outs[1][0]) and torch.isnan(outs[1][1]).all()


@pytest.mark.parametrize("wide", ["early key", "one group of every key", "one group of every third step", "all groups of every key"])
@pytest.mark.parametrize("T, D", [(1, 256), (2, 256), (1, 128), (3, 128), (1, 64)])
def test_small_values_beside_wide_ones(gpu_lib, T, D, wide):
    """60000 keys of values up to 15 * 2^-9, each e^-12 behind one key whose values are 0, in every group of 64 features that is
    not wide; `wide` groups or keys have values up to 15 * 100.  A group's small values are as exact as without them."""
    tsv, HQ, S = gpu_lib, 4, 60000
    gen = torch.Generator().manual_seed(T)
    pair = lambda s, b: torch.tensor([s, b]).half()  # noqa: E731
    k, v = ([torch.zeros(1, S + T, D // 2, dtype=torch.uint8), torch.zeros(1, S + T, D // 64, 2, dtype=torch.float16)] for _ in "kv")
    k[1][0, 0] = pair(0.0, 12.0 / D ** 0.5)
    v[0][:] = torch.randint(0, 256, v[0].shape, generator=gen)
    v[1][:] = pair(2.0 ** -9, 0.0)
    last = D // 64 - 1
    if wide == "early key":
        v[1][0, 20, last] = pair(100.0, -750.0)
    elif wide == "one group of every key":
        v[1][0, :, last] = pair(100.0, -750.0)
    elif wide == "one group of every third step":
        v[1][0, ::48, last] = pair(100.0, -750.0)
    else:
        v[1][:] = pair(100.0, -750.0)
    v[1][0, 0] = 0.0
    q = torch.ones(1, T, HQ, D).bfloat16()
    par = [list(range(-1, T - 1))]
    anc, _ = masks(tsv, par)
    o = torch.empty(1, T, HQ, D, dtype=torch.bfloat16, device=DEV)
    dev, qd = [[x[None].to(DEV) for x in y] for y in (k, v)], q.to(DEV)
    kv_len = torch.tensor([S + T], dtype=torch.int32, device=DEV)  # (a descriptor holds addresses)
    d = tsv.attn_desc([qd], [dev[0][0]], [dev[1][0]], [o], kv_len, anc, T=T, HQ=HQ,
                      HKV=1, D=D, kv_dtype=tsv.I4_G64, max_kv_len=S + T, k_scale=[dev[0][1]], v_scale=[dev[1][1]], splits=2)
    ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
    tsv.tree_verify_attention(d, ws)
    want, _ = ref_attention(q[0].double(), values(*k), values(*v), par[0], S)
    err = (o[0].double().cpu() - want).abs()
    # scores are exact in fp32; P times a scale is rounded once to fp16, 2^-11 of each term (all of one sign in a narrow group),
    # exp and the sums add 2^-20 of them; o is rounded to bf16 once.  Terms of a wide group: code * scale and bias apart,
    # each below 15 * 100 times the weight
    weight = 60000 * math.exp(-12) / (1 + 60000 * math.exp(-12))
    tol = (2.0 ** -8 + 2.0 ** -10) * want.abs()
    if wide in ("one group of every key", "all groups of every key"):
        g = slice(64 * last, None) if wide.startswith("one") else slice(None)
        tol[..., g] += 2.0 ** -10 * 2250 * weight
    elif D == 64 or wide.startswith("one"):
        tol[..., 64 * last:] += 2.0 ** -10 * 2250 * weight
    else:
        tol[..., 64 * last:] += 2.0 ** -10 * 2250 * math.exp(-12)
    assert (err <= tol).all(), (err / tol).max().item()


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("path", [0, 3, 4])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "i8"])
def test_a_query_row_that_is_not_finite_over_other_caches(gpu_lib, fmt, path, splits):
    """The same on the tensor-core kernels of the other formats, whose splits are merged by the same kernel."""
    tsv, B, T, HQ, HKV, D, S = gpu_lib, 1, 16, 24, 4, 256, 500
    gen = torch.Generator().manual_seed(path)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    if fmt == "i8":
        k, v = (torch.randint(-127, 128, (B, HKV, S + T, D), generator=gen, dtype=torch.int8).to(DEV) for _ in "kv")
        scales = dict(k_scale=[(0.01 * r(B, HKV, S + T).abs()).half()], v_scale=[(0.01 * r(B, HKV, S + T).abs()).half()])
    else:
        k, v = (r(B, HKV, S + T, D).to(torch.float16 if fmt == "f16" else torch.bfloat16) for _ in "kv")
        scales = {}
    kv_dtype = dict(f16=tsv.F16, bf16=tsv.BF16, i8=tsv.I8_SCALED)[fmt]
    anc, _ = masks(tsv, [random_tree(np.random.default_rng(1), T)])
    kv_len = torch.tensor([S + T], dtype=torch.int32, device=DEV)
    clean = r(B, T, HQ, D).bfloat16()

    def run(q):
        o = torch.full((B, T, HQ, D), 7.0, dtype=torch.bfloat16, device=DEV)
        d = tsv.attn_desc([q], [k], [v], [o], kv_len, anc, T=T, HQ=HQ, HKV=HKV, D=D, kv_dtype=kv_dtype, max_kv_len=S + T, splits=splits,
                          path=path, **scales)
        ws = torch.empty(max(tsv.attention_workspace_size(d), 16), dtype=torch.uint8, device=DEV)
        tsv.tree_verify_attention(d, ws)
        torch.cuda.synchronize()
        return o

    want = run(clean)
    for bad in (float("nan"), "one nan", 1e30):
        if fmt == "bf16" and bad == 1e30:
            continue  # within bf16: a finite, one-hot softmax
        q = clean.clone()
        if bad == "one nan":
            q[0, 5, 7, 9] = float("nan")
        else:
            q[0, 5, 7] = bad
        o = run(q)
        assert torch.isnan(o[0, 5, 7]).all(), bad
        o[0, 5, 7] = want[0, 5, 7]
        assert torch.equal(o, want), bad
