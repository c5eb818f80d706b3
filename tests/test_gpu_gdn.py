"""GPU parity of the recurrent calls (gated delta rule) against the fp64 recurrence.

Tolerances.  With unit keys and 0 <= beta <= 1 every step multiplies the state by e^g (I - beta k k^T), of norm at
most 1, so an error made at one token is never amplified by later ones: n tokens add up to n times what one token can
add.  One token's fp32 products over DK <= 128 terms, its decay (exp within 2 ulp, G from fp64) and its write are each
within (DK / 8 + 8) * 2^-24 of the magnitudes that enter it, M = max row norm of the state + max |v| along the run.
The tensor cores take the state, the writes u and the inner products as fp16, each within 2^-12 of its value, where they
only reach o, and as pairs within 2^-22 where they reach the state.  By Cauchy-Schwarz a product with the state is then
off by 2^-12 M; a sum over the block's earlier rows by 2^-11 W, W = max sum_j |k_i . k_j| |u_j| (and the same with q_i);
both once per row of the block, again never amplified.  o is rounded to bf16 once: 2^-8 |o|.
"""
import numpy as np
import pytest
import torch

from oracle import gdn as og

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(seed, L, B, rows, HK, HV, DK, DV, gate="usual"):
    """bf16 / fp32 inputs on the device; rows is (B, T) or (n,)."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = -torch.exp(n(L, *rows, HV) - 2.0)
    if gate == "none":
        g = torch.zeros_like(g)
    elif gate == "strong":
        g = g * 60.0
    elif gate == "forget":  # some tokens forget everything
        g[torch.rand(g.shape, generator=gen) < 0.2] = -float("inf")
    c = dict(q=n(L, *rows, HK, DK).bfloat16(), k=n(L, *rows, HK, DK).bfloat16(), v=n(L, *rows, HV, DV).bfloat16(), g=g,
             beta=torch.sigmoid(n(L, *rows, HV)), state=0.3 * n(L, B, HV, DV, DK))
    return {k: v.to(DEV) for k, v in c.items()}


def per(x, L):
    return [x[l] for l in range(L)]


def unit(x, eps):
    x = x.double()
    return x if eps == 0 else x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)


def ref_run(c, l, rows, parents, state, eps, scale):
    """fp64 recurrence over the rows `rows` (indices into the layer's rows), node i starting from parents[i]'s state
    (-1: `state`).  -> (o [n, HV, DV], states [n, HV, DV, DK], (M, W))."""
    HV = c["v"].shape[-2]
    flat = lambda x: x[l].reshape(-1, *x.shape[-2:])[rows]  # noqa: E731
    rep = HV // c["k"].shape[-2]
    q = unit(flat(c["q"]), eps).repeat_interleave(rep, dim=1)
    k = unit(flat(c["k"]), eps).repeat_interleave(rep, dim=1)
    v = flat(c["v"]).double()
    g, beta = (c[x][l].reshape(-1, HV)[rows].double() for x in ("g", "beta"))
    states, outs, us = [], [], []
    M = state.norm(dim=-1).max().item()
    for i, p in enumerate(parents):
        S = state.double() if p < 0 else states[p]
        S = torch.exp(g[i])[:, None, None] * S
        u = beta[i][:, None] * (v[i] - torch.einsum("hvk,hk->hv", S, k[i]))
        S = S + torch.einsum("hv,hk->hvk", u, k[i])
        states.append(S)
        us.append(u)
        outs.append(torch.einsum("hvk,hk->hv", S, q[i]) * scale)
        M = max(M, S.norm(dim=-1).max().item())
    n = len(parents)
    block = torch.arange(n, device=k.device) // 64
    near = (block[:, None] == block[None, :]).double()
    kt, u = k.transpose(0, 1), torch.stack(us).abs().transpose(0, 1)
    W = max(((torch.matmul(x.transpose(0, 1), kt.transpose(1, 2)).abs() * near) @ u).max().item() for x in (k, q))
    return torch.stack(outs), states, (M + v.abs().max().item(), W)


def close_o(got, want, MW, n, DK, scale):
    """Every element of o; M, W and the products' errors carry the factor scale (q is a unit row times it)."""
    M, W = MW
    rows = min(n, 64) + 1
    tol = 2.0 ** -8 * want.abs() + scale * (n * (DK / 8 + 8) * 2.0 ** -24 * M + rows * (2.0 ** -12 * M + 2.0 ** -11 * W))
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), (err - tol).max().item()
    # half a step of bf16 is at most 2^-8 of each value, so of the norm too; the fp16 errors mix signs
    assert err.norm() <= (2.0 ** -8 + 2.0 ** -10) * want.norm() + 1e-30


def close_state(got, want, MW, n, DK):
    M, W = MW
    err = (got.double() - want).abs().max().item()
    assert err <= n * ((DK / 8 + 8) * 2.0 ** -24 * M + 2.0 ** -22 * M + 2.0 ** -21 * W), (err, M, n)
    assert (got.double() - want).norm() <= 2.0 ** -18 * want.norm() + 1e-30  # far below the worst case: errors mix signs


def tree(rng, T, style):
    if style == "chain":
        return [-1] + list(range(T - 1))
    if style == "star":
        return [-1] + [0] * (T - 1)
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, T)]


def anc_of(tsv, parents):
    par = torch.tensor(np.array(parents, dtype=np.int32), device=DEV)
    B, T = par.shape
    anc = torch.zeros(B, T, dtype=torch.int64, device=DEV)
    tsv.tree_mask(par, anc, torch.zeros(B, T, dtype=torch.int32, device=DEV))
    return anc


def verify(tsv, c, parents, eps=1e-6, scale=0.0, anc=None):
    L = c["k"].shape[0]
    o = torch.full_like(c["v"], float("nan"))
    before = c["state"].clone()
    st = torch.zeros(4, dtype=torch.int32, device=DEV)
    d = tsv.gdn_desc(*(per(c[x], L) for x in ("q", "k", "v", "g", "beta", "state")), o=per(o, L), norm_eps=eps, scale=scale)
    tsv.gdn_tree_verify(d, anc_of(tsv, parents) if anc is None else anc, dev_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0, 0, 0]
    assert torch.equal(c["state"], before)
    return o


def check_verify(tsv, c, parents, eps=1e-6, scale=0.0):
    o = verify(tsv, c, parents, eps, scale)
    L, B, T = c["k"].shape[:3]
    sc = scale or c["k"].shape[-1] ** -0.5
    for l in range(L):
        for b in range(B):
            want, _, M = ref_run(c, l, slice(b * T, (b + 1) * T), parents[b], c["state"][l, b], eps, sc)
            close_o(o[l, b], want, M, T, c["k"].shape[-1], sc)


@pytest.mark.parametrize("style", ["random", "chain", "star"])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 49, 63, 64])
def test_tree_verify_sizes(gpu_lib, T, style):
    rng = np.random.default_rng(T)
    check_verify(gpu_lib, case(T, 1, 2, (2, T), 2, 6, 128, 128), [tree(rng, T, style) for _ in range(2)])


@pytest.mark.parametrize("DK, DV", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("HK, HV", [(1, 1), (2, 8), (5, 5)])
@pytest.mark.parametrize("T", [4, 20, 64])
def test_tree_verify_heads(gpu_lib, T, HK, HV, DK, DV):
    rng = np.random.default_rng(T + DK)
    check_verify(gpu_lib, case(T, 3, 1, (1, T), HK, HV, DK, DV), [tree(rng, T, "random")])


@pytest.mark.parametrize("gate", ["none", "strong", "forget"])
@pytest.mark.parametrize("T", [3, 16, 64])
def test_tree_verify_gates(gpu_lib, T, gate):
    rng = np.random.default_rng(T)
    check_verify(gpu_lib, case(T, 1, 2, (2, T), 1, 2, 128, 128, gate), [tree(rng, T, s) for s in ("random", "chain")])


@pytest.mark.parametrize("T", [3, 40])
def test_tree_verify_without_norms_and_with_a_scale(gpu_lib, T):
    c = case(T, 1, 1, (1, T), 2, 2, 128, 128)
    for x in "qk":  # already unit rows, rounded to bf16 (norm within 2^-8 of 1)
        c[x] = unit(c[x], 1e-6).bfloat16()
    c["k"] = c["k"] * 0.5
    check_verify(gpu_lib, c, [tree(np.random.default_rng(1), T, "random")], eps=0.0, scale=0.25)


@pytest.mark.parametrize("T", [5, 19])
def test_tree_verify_beyond_fp16(gpu_lib, T):
    """Keys far from unit length with large writes: values leave fp16's range (not fp32's) within a few nodes, and rows
    of the state 2^60 apart."""
    c = case(T, 1, 1, (1, T), 1, 2, 128, 128)
    c["k"] = c["k"] * 8.0
    c["state"][:, :, :, 1::2] *= 2.0 ** -60
    c["v"][..., 1::2] *= 2.0 ** -60
    c["g"][:] = 0.0
    par = [tree(np.random.default_rng(T), T, "random")]
    depth = max(len(_path(par[0], i)) for i in range(T))
    o = verify(gpu_lib, c, par, eps=0.0)
    want, states, _ = ref_run(c, 0, slice(0, T), par[0], c["state"][0, 0], 0.0, 128 ** -0.5)
    for half in (slice(0, None, 2), slice(1, None, 2)):
        x, y = o[0, 0, :, :, half].double(), want[..., half]
        # each step multiplies what came before by up to beta |k|^2 < 10^5; errors relative to a path's largest values
        assert (x - y).norm() <= (2.0 ** -8 + 2.0 ** -10) * y.norm()
    assert depth > 3 and want.abs().max() > 65504


@pytest.mark.parametrize("T", [6, 16, 30, 64])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta", "inf"])
def test_a_nan_stays_with_its_node_and_descendants(gpu_lib, T, what):
    rng = np.random.default_rng(T)
    par = tree(rng, T, "random")
    j = T // 3
    below = [i for i in range(T) if j in _path(par, i)]
    c = case(T, 1, 1, (1, T), 1, 2, 128, 128)
    clean = verify(gpu_lib, c, [par])
    x = c["v" if what == "inf" else what]
    x[0, 0, j] = float("inf") if what == "inf" else float("nan")
    o = verify(gpu_lib, c, [par])
    rest = [i for i in range(T) if i not in below]
    assert torch.isfinite(o[0, 0, rest]).all()
    # the clean run's values, up to the two ways a tree may be computed
    err = (o[0, 0, rest].double() - clean[0, 0, rest].double()).abs()
    assert (err <= 2.0 ** -7 * clean[0, 0, rest].double().abs() + 1e-3).all()
    assert not torch.isfinite(o[0, 0, j]).any()


def _path(par, i):
    out = [i]
    while par[out[-1]] >= 0:
        out.append(par[out[-1]])
    return out


@pytest.mark.parametrize("T", [5, 33])
def test_ancestor_bits_at_or_above_a_node_are_ignored(gpu_lib, T):
    rng = np.random.default_rng(T)
    par = tree(rng, T, "random")
    c = case(T, 1, 1, (1, T), 1, 1, 128, 128)
    anc = anc_of(gpu_lib, [par])
    high = torch.tensor([[-(1 << i) if i < 63 else -(1 << 63) for i in range(T)]], device=DEV)
    assert torch.equal(verify(gpu_lib, c, [par]), verify(gpu_lib, c, [par], anc=anc | high))


def commit(tsv, c, path, path_len, state_out=None, st=None):
    L = c["k"].shape[0]
    st = torch.zeros(4, dtype=torch.int32, device=DEV) if st is None else st
    d = tsv.gdn_desc(None, *(per(c[x], L) for x in ("k", "v", "g", "beta", "state")),
                     state_out=None if state_out is None else per(state_out, L))
    tsv.gdn_commit(d, torch.tensor(path, dtype=torch.int32, device=DEV), torch.tensor(path_len, dtype=torch.int32, device=DEV),
                   dev_status=st)
    torch.cuda.synchronize()
    return st


@pytest.mark.parametrize("DK, DV, HK, HV", [(128, 128, 2, 6), (64, 64, 1, 2), (64, 128, 3, 3), (128, 64, 1, 4)])
@pytest.mark.parametrize("T, paths", [(1, [[0]]), (16, [[0, 2, 5, 11, 15], [0], [0, 1, 2, 3]]), (64, [list(range(64)), [0, 63]])])
def test_commit(gpu_lib, T, paths, DK, DV, HK, HV):
    B = len(paths)
    c = case(T, 2, B, (B, T), HK, HV, DK, DV)
    padded, lens = [p + [-1] * (T - len(p)) for p in paths], [len(p) for p in paths]
    out = torch.full_like(c["state"], float("nan"))
    before = c["state"].clone()
    assert commit(gpu_lib, c, padded, lens, out).tolist() == [0, 0, 0, 0]
    assert torch.equal(c["state"], before)
    for l in range(2):
        for b, p in enumerate(paths):
            _, S, M = ref_run(c, l, [b * T + j for j in p], list(range(-1, len(p) - 1)), c["state"][l, b], 1e-6, 1.0)
            close_state(out[l, b], S[-1], M, len(p), DK)
    assert commit(gpu_lib, c, padded, lens).tolist() == [0, 0, 0, 0]  # in place
    assert torch.equal(c["state"], out)


@pytest.mark.parametrize("path, n", [([1, 2, 3, 3], 2), ([0, 2, 2, 3], 3), ([0, 3, 1, 2], 3), ([0, 4, -1, -1], 2), ([0, 1, 2, 3], 0),
                                     ([0, 1, 2, 3], 5), ([0, -1, 2, 3], 3), ([0, 1, 2, 3], -7), ([0, 1 << 30, 2, 3], 2)])
def test_commit_reports_a_bad_path_and_leaves_that_sequence(gpu_lib, path, n):
    c = case(1, 1, 2, (2, 4), 1, 2, 128, 128)
    out = torch.full_like(c["state"], 7.0)
    st = commit(gpu_lib, c, [[0, 1, 2, 3], path], [2, n], out)
    assert st.tolist()[:2] == [gpu_lib.DEV_BAD_PATH, 1]
    assert (out[:, 1] == 7.0).all()
    _, S, M = ref_run(c, 0, [0, 1], [-1, 0], c["state"][0, 0], 1e-6, 1.0)
    close_state(out[0, 0], S[-1], M, 2, 128)


def scan(tsv, c, cu, max_len, state_out=None, o=None, st=None, eps=1e-6, scale=0.0):
    L = c["k"].shape[0]
    o = torch.full_like(c["v"], -77.0) if o is None else o
    st = torch.zeros(4, dtype=torch.int32, device=DEV) if st is None else st
    d = tsv.gdn_desc(*(per(c[x], L) for x in ("q", "k", "v", "g", "beta", "state")), o=per(o, L),
                     state_out=None if state_out is None else per(state_out, L), norm_eps=eps, scale=scale)
    tsv.gdn_scan(d, torch.tensor(cu, dtype=torch.int32, device=DEV), max_len=max_len, dev_status=st)
    torch.cuda.synchronize()
    return o, st


def check_scan(tsv, c, lens, max_len=None, lead=0, eps=1e-6, scale=0.0, layers=None):
    """lens: tokens per sequence; `lead` rows ahead of the first sequence and whatever follows the last are no one's."""
    DK = c["k"].shape[-1]
    cu = [lead]
    for n in lens:
        cu.append(cu[-1] + n)
    out = torch.full_like(c["state"], float("nan"))
    before = c["state"].clone()
    o, st = scan(tsv, c, cu, max(lens) if max_len is None else max_len, out, eps=eps, scale=scale)
    assert st.tolist() == [0, 0, 0, 0]
    assert torch.equal(c["state"], before)
    assert (o[:, :lead] == -77.0).all() and (o[:, cu[-1]:] == -77.0).all()
    sc = scale or DK ** -0.5
    for l in range(c["k"].shape[0]):
        for b, n in enumerate(lens):
            if n == 0:
                assert torch.equal(out[l, b], c["state"][l, b])
                continue
            want, S, M = ref_run(c, l, slice(cu[b], cu[b + 1]), list(range(-1, n - 1)), c["state"][l, b], eps, sc)
            close_o(o[l, cu[b]:cu[b + 1]], want, M, n, DK, sc)
            close_state(out[l, b], S[-1], M, n, DK)
    return o, out


@pytest.mark.parametrize("lens", [[1], [1, 1, 1, 1, 1], [0, 1, 0], [2], [3, 7, 8], [9], [16], [17, 1, 0, 33], [63], [64], [65],
                                  [127, 128, 129], [200, 0, 5, 64, 1, 190], [500]])
def test_scan_lengths(gpu_lib, lens):
    total = sum(lens) + 5
    check_scan(gpu_lib, case(total, 1, len(lens), (total,), 2, 6, 128, 128), lens, lead=2)


@pytest.mark.parametrize("DK, DV", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("HK, HV", [(1, 1), (2, 8), (5, 5)])
@pytest.mark.parametrize("lens", [[1, 1], [70, 3, 130]])
def test_scan_heads(gpu_lib, lens, HK, HV, DK, DV):
    check_scan(gpu_lib, case(7, 2, len(lens), (sum(lens),), HK, HV, DK, DV), lens)


@pytest.mark.parametrize("gate", ["none", "strong", "forget"])
@pytest.mark.parametrize("lens", [[4, 1], [150, 64]])
def test_scan_gates(gpu_lib, lens, gate):
    check_scan(gpu_lib, case(8, 1, 2, (sum(lens),), 1, 3, 128, 128, gate), lens)


def test_scan_with_equal_keys_and_full_writes(gpu_lib):
    """Keys all alike and beta = 1: each token overwrites what the one before wrote, the system's worst conditioning."""
    c = case(9, 1, 1, (200,), 1, 2, 128, 128, "none")
    c["k"][:] = c["k"][:, :1]
    c["beta"][:] = 1.0
    check_scan(gpu_lib, c, [200])


def test_scan_without_norms_and_with_a_scale(gpu_lib):
    c = case(10, 1, 2, (150,), 2, 2, 128, 128)
    for x in "qk":
        c[x] = unit(c[x], 1e-6).bfloat16() * 0.5
    check_scan(gpu_lib, c, [131, 19], eps=0.0, scale=0.25)


@pytest.mark.parametrize("lens", [[5, 3], [150, 70]])
def test_a_max_len_above_the_lengths(gpu_lib, lens):
    check_scan(gpu_lib, case(11, 1, 2, (300,), 1, 2, 128, 128), lens, max_len=300)


def test_scan_in_parts_is_the_whole_scan(gpu_lib):
    c = case(12, 1, 1, (200,), 1, 4, 128, 128)
    o, out = check_scan(gpu_lib, c, [200])
    for parts in ([64, 136], [1, 199], [100, 3, 97]):
        state, at, rows = c["state"].clone(), 0, []
        for n in parts:
            part = {x: c[x][:, at:at + n].contiguous() for x in ("q", "k", "v", "g", "beta")}
            part["state"] = state
            rows.append(scan(gpu_lib, part, [0, n], n)[0])  # in place
            at += n
        want, S, M = ref_run(c, 0, slice(0, 200), list(range(-1, 199)), c["state"][0, 0], 1e-6, 128 ** -0.5)
        close_o(torch.cat(rows, dim=1)[0], want, M, 200, 128, 128 ** -0.5)
        close_state(state[0, 0], S[-1], M, 200, 128)


@pytest.mark.parametrize("long", [False, True])
def test_scan_reports_bad_lengths_and_leaves_those_sequences(gpu_lib, long):
    """Descending, beyond the rows, below zero, longer than max_len: that sequence is left, the others are computed."""
    n, top = (90, 90) if long else (4, 4)
    rows = 2 * n
    c = case(13, 1, 3, (rows,), 1, 2, 128, 128)
    for cu, bad, max_len in (([0, n, n - 1, rows], 1, max(n + 1, top)), ([0, n, 2 * n, 2 * n + 1], 2, top), ([-1, n, n, n], 0, n + 1),
                             ([0, n, n + n, n + n], 0, n - 1)):
        out = torch.full_like(c["state"], 7.0)
        o, st = scan(gpu_lib, c, cu, min(max_len, rows), out)
        assert st.tolist()[0] == gpu_lib.DEV_BAD_SEQ_LEN
        assert (out[:, bad] == 7.0).all()
        for b in range(3):
            if cu[b] >= 0 and 0 < cu[b + 1] - cu[b] <= max_len and cu[b + 1] <= rows and b != bad:
                _, S, M = ref_run(c, 0, slice(cu[b], cu[b + 1]), list(range(-1, cu[b + 1] - cu[b] - 1)), c["state"][0, b], 1e-6, 1.0)
                close_state(out[0, b], S[-1], M, cu[b + 1] - cu[b], 128)


@pytest.mark.parametrize("n, j", [(5, 2), (150, 70), (150, 149), (150, 64)])
@pytest.mark.parametrize("what", ["v", "k", "g"])
def test_a_nan_reaches_later_tokens_only(gpu_lib, n, j, what):
    c = case(14, 1, 2, (2 * n,), 1, 2, 128, 128)
    clean, _ = scan(gpu_lib, c, [0, n, 2 * n], n, torch.empty_like(c["state"]))
    c[what][0, j] = float("nan")
    o, _ = scan(gpu_lib, c, [0, n, 2 * n], n, torch.empty_like(c["state"]))
    for rows in (slice(0, j), slice(n, 2 * n)):
        assert torch.isfinite(o[0, rows]).all()
        err = (o[0, rows].double() - clean[0, rows].double()).abs()
        assert (err <= 2.0 ** -7 * clean[0, rows].double().abs() + 1e-3).all()
    assert not torch.isfinite(o[0, j:n]).any()


def test_a_nan_in_one_value_feature_stays_there(gpu_lib):
    c = case(15, 1, 1, (150,), 1, 1, 128, 128)
    clean, s0 = scan(gpu_lib, c, [0, 150], 150, torch.empty_like(c["state"]))
    c["v"][0, 20, 0, 5] = float("nan")
    out = torch.empty_like(c["state"])
    o, _ = scan(gpu_lib, c, [0, 150], 150, out)
    keep = [f for f in range(128) if f != 5]
    assert torch.isfinite(o[0, :, 0][:, keep]).all() and torch.isfinite(out[0, 0, 0][keep]).all()
    assert torch.isfinite(o[0, :20]).all() and torch.isnan(o[0, 20:, 0, 5]).all()


def test_streams_and_graphs(gpu_lib):
    """The three calls on a side stream, and captured twice over different buffers and replayed in turn."""
    L, B, T = 2, 2, 12
    rng = np.random.default_rng(3)
    par = [tree(rng, T, "random") for _ in range(B)]
    anc = anc_of(gpu_lib, par)
    path = torch.tensor([[0, 2, 7] + [-1] * (T - 3), [0] + [-1] * (T - 1)], dtype=torch.int32, device=DEV)
    plen = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 100, 130], dtype=torch.int32, device=DEV)
    sets = []
    for seed in (1, 2):
        t, s = case(seed, L, B, (B, T), 2, 4, 128, 128), case(seed + 9, L, B, (130,), 2, 4, 128, 128)
        o, so = torch.empty_like(t["v"]), torch.empty_like(s["v"])
        t_out, s_out = torch.empty_like(t["state"]), torch.empty_like(s["state"])
        f = lambda c, **kw: gpu_lib.gdn_desc(*(per(c[x], L) for x in ("q", "k", "v", "g", "beta", "state")),  # noqa: E731
                                             **{k: per(v, L) for k, v in kw.items()})
        dt, ds = f(t, o=o, state_out=t_out), f(s, o=so, state_out=s_out)
        sets.append((t, s, (o, so, t_out, s_out), dt, ds))

    def calls(dt, ds):
        gpu_lib.gdn_tree_verify(dt, anc)
        gpu_lib.gdn_commit(dt, path, plen)
        gpu_lib.gdn_scan(ds, cu, max_len=100)

    want = []
    for _, _, outs, dt, ds in sets:
        calls(dt, ds)
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs])
        for x in outs:
            x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(sets[0][3], sets[0][4])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(sets[0][2], want[0]))
    graphs = []
    for _, _, outs, dt, ds in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(dt, ds)
        graphs.append(g)
    for _ in range(2):
        for s, w, g in zip(sets, want, graphs):
            for x in s[2]:
                x.zero_()
            g.replay()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(s[2], w))


def test_the_binding_refuses_the_wrong_layout(gpu_lib):
    c, p = case(1, 1, 1, (1, 4), 1, 1, 128, 128), case(1, 1, 1, (4,), 1, 1, 128, 128)
    f = lambda c: gpu_lib.gdn_desc(*(per(c[x], 1) for x in ("q", "k", "v", "g", "beta", "state")), o=per(c["v"].clone(), 1))  # noqa: E731
    cu = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="packed"):
        gpu_lib.gdn_scan(f(c), cu, max_len=4)
    with pytest.raises(ValueError, match="tree block"):
        gpu_lib.gdn_tree_verify(f(p), torch.zeros(1, 4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        gpu_lib.gdn_desc(*(per(c[x], 1) for x in ("q", "k", "v", "g", "beta")), [c["state"][0].transpose(-1, -2)])
    with pytest.raises(ValueError, match="cu_len"):
        gpu_lib.gdn_scan(f(p), cu[:1], max_len=4)


def test_small_tree_against_the_numpy_oracle(gpu_lib):
    c = case(4, 1, 1, (1, 7), 2, 4, 64, 64)
    par = [-1, 0, 0, 1, 1, 2, 2]
    o = verify(gpu_lib, c, [par])
    n = {x: c[x][0, 0].double().cpu().numpy() for x in ("q", "k", "v", "g", "beta", "state")}
    want = og.tree_verify(n["q"], n["k"], n["v"], n["g"], n["beta"], n["state"], par)
    assert np.abs(o[0, 0].double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-4


# ----------------------------------------------------------------------------- the grids that large batches take
@pytest.mark.parametrize("T", [5, 16, 20, 48, 64])
@pytest.mark.parametrize("HK, HV", [(4, 4), (2, 4), (2, 6), (2, 8), (1, 5)])
def test_tree_verify_of_large_batches(gpu_lib, T, HK, HV):
    """Enough heads that the value heads of one key head share a CTA (two, three or four of them; five do not split);
    one head's operands leave fp16's range, one holds a NaN: the others of their CTA are as without them."""
    L, B = 40, 16
    rng = np.random.default_rng(T)
    par = [tree(rng, T, "random") for _ in range(B)]
    c = case(T, L, B, (B, T), HK, HV, 128, 128)
    clean = verify(gpu_lib, c, par)
    for l, b in ((0, 0), (L - 1, B - 1), (17, 5)):
        want, _, M = ref_run(c, l, slice(b * T, (b + 1) * T), par[b], c["state"][l, b], 1e-6, 128 ** -0.5)
        close_o(clean[l, b], want, M, T, 128, 128 ** -0.5)
    c["v"][3, 2, T - 1, HV - 1] = float("nan")
    c["v"][3, 2, :, 0, 7] *= 1e30
    c["state"][3, 2, 0, 9] = 1e25
    o = verify(gpu_lib, c, par)
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[3, 2, :, 0] = False
    keep[3, 2, :, HV - 1] = False
    assert torch.equal(o[keep], clean[keep])
    assert not torch.isfinite(o[3, 2, T - 1, HV - 1]).any()
    if HV > 1:  # features of very different size in one head: each is as exact as alone
        want, _, _ = ref_run(c, 3, slice(2 * T, 3 * T), par[2], c["state"][3, 2], 1e-6, 128 ** -0.5)
        for f in (7, 9, 20):
            x, y = o[3, 2, :, 0, f].double(), want[:, 0, f]
            assert (x - y).norm() <= (2.0 ** -8 + 2.0 ** -9) * y.norm()


@pytest.mark.parametrize("DK, DV", [(64, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("what", ["clean", "v", "k", "wide"])
def test_scan_of_large_batches(gpu_lib, what, DK, DV):
    """Whole heads per CTA (many of them), sequences started in another order than theirs, bad values in one."""
    lens = [70, 0, 200, 17, 64, 129, 33]
    c = case(21, 1, len(lens), (sum(lens) + 4,), 4, 16, DK, DV)
    at = lens[0] + 100  # token 100 of the third sequence
    if what in ("v", "k"):
        clean, s0 = scan(gpu_lib, c, np.cumsum([2] + lens).tolist(), max(lens), torch.empty_like(c["state"]))
        c[what][0, 2 + at, 1] = float("nan")
        o, _ = scan(gpu_lib, c, np.cumsum([2] + lens).tolist(), max(lens), torch.empty_like(c["state"]))
        hit = torch.zeros(o.shape[1:3], dtype=torch.bool, device=DEV)
        heads = [1] if what == "v" else [4, 5, 6, 7]
        hit[2 + at:2 + lens[0] + lens[2], heads] = True
        assert not torch.isfinite(o[0][hit]).any()
        # the chunk ahead of the NaN is done again token by token: the same values up to bf16's rounding of either
        x, y = o[0][~hit].double(), clean[0][~hit].double()
        assert ((x - y).abs() <= 2.0 ** -7 * y.abs() + 1e-3).all()
        return
    if what == "wide":  # v's features 2^80 apart
        c["v"][..., ::2] *= 2.0 ** -80
        c["state"][:, :, :, ::2] *= 2.0 ** -80
        cu = np.cumsum([2] + lens).tolist()
        out = torch.empty_like(c["state"])
        o, st = scan(gpu_lib, c, cu, max(lens), out)
        want, S, _ = ref_run(c, 0, slice(cu[2], cu[3]), list(range(-1, lens[2] - 1)), c["state"][0, 2], 1e-6, DK ** -0.5)
        for half in (slice(0, None, 2), slice(1, None, 2)):
            assert (o[0, cu[2]:cu[3]][..., half].double() - want[..., half]).norm() <= (2.0 ** -8 + 2.0 ** -9) * want[..., half].norm()
            assert (out[0, 2][:, half].double() - S[-1][:, half]).norm() <= 2.0 ** -18 * S[-1][:, half].norm()
        return
    check_scan(gpu_lib, c, lens, lead=2)


def test_scan_of_more_sequences_than_are_sorted(gpu_lib):
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 300)]
    check_scan(gpu_lib, case(22, 1, 300, (sum(lens),), 1, 1, 128, 128), lens)


def test_scan_token_by_token_of_many_heads(gpu_lib):
    """Up to 17 tokens a call go token by token when there are this many heads."""
    lens = [17] * 20 + [12, 1, 0, 16, 9, 17]
    check_scan(gpu_lib, case(27, 1, len(lens), (sum(lens),), 16, 48, 64, 64), lens)


@pytest.mark.parametrize("lens", [[0] * 299 + [500], [int(x) for x in np.random.default_rng(5).integers(0, 200, 384)],
                                  [int(x) for x in np.random.default_rng(6).integers(0, 200, 385)],
                                  [65, 64, 128, 129, 0, 65, 64, 129, 1, 192, 193, 65], [64] * 33 + [65], [300, 0]])
def test_scan_in_the_order_of_lengths(gpu_lib, lens):
    """Every sequence is taken by exactly one CTA per head, whatever the order: many equal ones, a long one at the end,
    as many as there are threads, one more."""
    B = len(lens)
    check_scan(gpu_lib, case(25, 1, B, (sum(lens) + 3,), 1, 1, 64, 64), lens, lead=1)
    c = case(26, 1, B, (sum(lens),), 1, 2, 128, 128)
    cu = np.cumsum([0] + lens).tolist()
    bad = int(np.argmax(lens))  # the longest does not fit max_len: reported, the others as they are
    out, ref = torch.full_like(c["state"], 7.0), torch.full_like(c["state"], 7.0)
    scan(gpu_lib, c, cu, max(lens), ref)
    _, st = scan(gpu_lib, c, cu, max(lens) - 1, out)
    assert st.tolist()[0] == gpu_lib.DEV_BAD_SEQ_LEN
    for b in range(B):
        if lens[b] == max(lens):
            assert (out[:, b] == 7.0).all()
        else:
            assert torch.equal(out[:, b], ref[:, b])
    assert st.tolist()[1] < B and lens[st.tolist()[1]] == lens[bad]


def test_scan_beyond_fp16(gpu_lib):
    """Keys far from unit length: the recurrence grows beyond fp16's range, token by token in fp32 then, and stays exact
    where it still is finite."""
    for n in (40, 150):
        c = case(23, 1, 1, (n,), 1, 2, 128, 128, "none")
        c["k"] = c["k"] * (0.5 if n == 40 else 0.35)
        o, st = scan(gpu_lib, c, [0, n], n, torch.empty_like(c["state"]), eps=0.0)
        want, S, _ = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 0.0, 128 ** -0.5)
        assert want.abs().max() > 65504
        # every step multiplies a direction by up to |1 - beta |k|^2|: errors grow as the values do
        assert (o[0].double() - want).norm() <= (2.0 ** -8 + 2.0 ** -10) * want.norm()


def test_scan_without_rows(gpu_lib):
    c = case(24, 2, 3, (0,), 1, 2, 128, 128)
    out = torch.full_like(c["state"], 7.0)
    o, st = scan(gpu_lib, c, [0, 0, 0, 0], 0, out)
    assert st.tolist() == [0, 0, 0, 0] and torch.equal(out, c["state"])


def test_scan_rows_beyond_32_bits(gpu_lib):
    """Rows whose v and o lie past 2^31 bytes."""
    HV, rows, n = 64, (1 << 31) // (64 * 128 * 2) + 300, 100
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
    c = dict(q=torch.empty(1, rows, 1, 128, dtype=torch.bfloat16, device=DEV), k=torch.empty(1, rows, 1, 128, dtype=torch.bfloat16, device=DEV),
             v=torch.empty(1, rows, HV, 128, dtype=torch.bfloat16, device=DEV), g=torch.empty(1, rows, HV, device=DEV),
             beta=torch.empty(1, rows, HV, device=DEV), state=0.3 * r(1, 1, HV, 128, 128))
    at = rows - n
    c["q"][0, at:], c["k"][0, at:], c["v"][0, at:] = r(n, 1, 128).bfloat16(), r(n, 1, 128).bfloat16(), r(n, HV, 128).bfloat16()
    c["g"][0, at:], c["beta"][0, at:] = -r(n, HV).abs(), torch.sigmoid(r(n, HV))
    o = torch.empty_like(c["v"])
    out = torch.empty_like(c["state"])
    for m in (n, 5):  # in chunks, token by token
        scan(gpu_lib, c, [rows - m, rows], m, out, o=o)
        want, S, M = ref_run(c, 0, slice(rows - m, rows), list(range(-1, m - 1)), c["state"][0, 0], 1e-6, 128 ** -0.5)
        close_o(o[0, rows - m:], want, M, m, 128, 128 ** -0.5)
        close_state(out[0, 0], S[-1], M, m, 128)


@pytest.mark.parametrize("T", [1, 9, 64])
def test_two_calls_at_once(gpu_lib, T):
    """The calls on two streams at a time, over their own outputs, give what they give one after the other."""
    rng = np.random.default_rng(T)
    L, B = 4, 8
    par = [tree(rng, T, "random") for _ in range(B)]
    anc = anc_of(gpu_lib, par)
    cu = torch.arange(0, 30 * (B + 1), 30, dtype=torch.int32, device=DEV)
    t, s = case(1, L, B, (B, T), 2, 8, 128, 128), case(2, L, B, (30 * B,), 2, 8, 128, 128)
    outs = [[torch.empty_like(t["v"]), torch.empty_like(s["v"]), torch.empty_like(s["state"])] for _ in range(3)]

    def calls(x):
        gpu_lib.gdn_tree_verify(gpu_lib.gdn_desc(*(per(t[y], L) for y in ("q", "k", "v", "g", "beta", "state")), o=per(x[0], L)), anc)
        gpu_lib.gdn_scan(gpu_lib.gdn_desc(*(per(s[y], L) for y in ("q", "k", "v", "g", "beta", "state")), o=per(x[1], L),
                                          state_out=per(x[2], L)), cu, max_len=30)

    calls(outs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for st, x in zip(streams, outs[1:]):
            with torch.cuda.stream(st):
                calls(x)
    torch.cuda.synchronize()
    for x in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, outs[0]))


@pytest.mark.parametrize("scale", [1e-9, 2.0 ** -20, 1e-4, 3e4, 1e12])
@pytest.mark.parametrize("empty", [False, True])
def test_any_scale(gpu_lib, scale, empty):
    """o is as exact under a small or large scale as under the usual one, also where it comes from the block's own writes
    alone (empty states)."""
    rng = np.random.default_rng(1)
    for T in (3, 16, 40, 64):
        c = case(T, 1, 2, (2, T), 2, 4, 128, 128)
        if empty:
            c["state"].zero_()
        check_verify(gpu_lib, c, [tree(rng, T, "random") for _ in range(2)], scale=scale)
    c = case(5, 1, 2, (150,), 2, 4, 128, 128)
    if empty:
        c["state"].zero_()
    check_scan(gpu_lib, c, [100, 50], scale=scale)


@pytest.mark.parametrize("mq, mk", [(2.0 ** -12, 1.0), (2.0 ** -7, 2.0 ** -7), (2.0 ** -10, 2.0 ** -10), (2.0 ** -30, 2.0 ** -4), (1.0, 2.0 ** -12),
                                    (200.0, 1.0), (2000.0, 1.0)])
def test_rows_far_from_unit_length(gpu_lib, mq, mk):
    """norm_eps 0 with short or long rows of q and k over empty states: o is as small as their product, as exact as ever
    relative to itself."""
    rng = np.random.default_rng(2)
    for T in (5, 40, 64):
        c = case(T, 1, 1, (1, T), 1, 2, 128, 128)
        c["q"], c["k"] = unit(c["q"], 1e-6).bfloat16() * mq, unit(c["k"], 1e-6).bfloat16() * mk
        c["state"].zero_()
        par = tree(rng, T, "random")
        o = verify(gpu_lib, c, [par], eps=0.0, scale=1.0)
        want, _, _ = ref_run(c, 0, slice(0, T), par, c["state"][0, 0], 0.0, 1.0)
        # a bf16 rounding and fp16 operands (2^-12 each, mixing signs), relative to o itself
        assert (o[0, 0].double() - want).norm() <= (2.0 ** -8 + 2.0 ** -10) * want.norm()
    c = case(6, 1, 1, (150,), 1, 2, 128, 128)
    c["q"], c["k"] = unit(c["q"], 1e-6).bfloat16() * mq, unit(c["k"], 1e-6).bfloat16() * mk
    c["state"].zero_()
    out = torch.empty_like(c["state"])
    o, _ = scan(gpu_lib, c, [0, 150], 150, out, eps=0.0, scale=1.0)
    want, S, _ = ref_run(c, 0, slice(0, 150), list(range(-1, 149)), c["state"][0, 0], 0.0, 1.0)
    assert (o[0].double() - want).norm() <= (2.0 ** -8 + 2.0 ** -10) * want.norm()
    assert (out[0, 0].double() - S[-1]).norm() <= 2.0 ** -18 * S[-1].norm()  # as close_state's bound on the norm


# ----------------------------------------------------------------------------- values of very different size in one block
def rows_close(got, want, rel=2.0 ** -8 + 2.0 ** -9):
    """Every row (last axis) relative to its own norm: bf16's rounding is within 2^-8 of each value, so of the norm."""
    err, size = (got.double() - want).norm(dim=-1), want.norm(dim=-1)
    assert (err <= rel * size + 1e-37).all(), (err / size.clamp_min(1e-37)).max().item()


def within_o(got, want, MW, n, DK, scale):
    """close_o's bound per element, of the module's derivation, without the one on the norm."""
    M, W = MW
    tol = 2.0 ** -8 * want.abs() + scale * (n * (DK / 8 + 8) * 2.0 ** -24 * M + (min(n, 64) + 1) * (2.0 ** -12 * M + 2.0 ** -11 * W))
    assert ((got.double() - want).abs() <= tol).all()


def within_state(got, want, MW, n, DK):
    """close_state's bound per element."""
    M, W = MW
    assert (got.double() - want).abs().max() <= n * ((DK / 8 + 8) * 2.0 ** -24 * M + 2.0 ** -22 * M + 2.0 ** -21 * W)


def enlarge(x, power, what):
    """Rows x [HV, DV] of one node or token: all of it, or one value feature of the last head, 2^power times as large."""
    if what == "row":
        x *= 2.0 ** power
    else:
        x[-1, 37] = 1.5 * 2.0 ** power


@pytest.mark.parametrize("what", ["row", "feature"])
@pytest.mark.parametrize("power", [10, 16, 19, 22, 24, 26, 28, 31, 60, 100])
@pytest.mark.parametrize("T, j", [(2, 1), (4, 2), (16, 9), (17, 1), (40, 30), (64, 5), (64, 63)])
def test_a_large_value_stays_with_its_node_and_descendants(gpu_lib, T, j, power, what):
    """One node's v 2^power times the others': nodes that do not see it are as exact as without it."""
    par = tree(np.random.default_rng(T + j), T, "random")
    below = [i for i in range(T) if j in _path(par, i)]
    rest = [i for i in range(T) if i not in below]
    for fresh in (False, True):
        c = case(T + power, 1, 1, (1, T), 1, 3, 128, 128)
        if fresh:
            c["state"].zero_()
        want, _, MW = ref_run(c, 0, slice(0, T), par, c["state"][0, 0], 1e-6, 128 ** -0.5)
        enlarge(c["v"][0, 0, j], power, what)
        o = verify(gpu_lib, c, [par])[0, 0]
        close_o(o[rest], want[rest], MW, T, 128, 128 ** -0.5)
        rows_close(o[rest], want[rest])
        if what == "feature":
            rows_close(o[rest, -1, 37].unsqueeze(0), want[rest, -1, 37].unsqueeze(0))
            others = [f for f in range(128) if f != 37]
            close_o(o[..., others], want[..., others], MW, T, 128, 128 ** -0.5)
        # what sees it is as exact as the largest values it is summed from
        want, _, MW = ref_run(c, 0, slice(0, T), par, c["state"][0, 0], 1e-6, 128 ** -0.5)
        within_o(o[below], want[below], MW, T, 128, 128 ** -0.5)


@pytest.mark.parametrize("power", [-10, -20, -24, -26, -30, -40, -90])
@pytest.mark.parametrize("T", [2, 16, 33, 64])
def test_a_small_root_before_larger_nodes(gpu_lib, T, power):
    """The root of an empty state sees itself alone: its o is exact relative to its own size."""
    par = tree(np.random.default_rng(T), T, "random")
    c = case(T, 1, 1, (1, T), 1, 2, 128, 128)
    c["state"].zero_()
    c["v"][0, 0, 0] *= 2.0 ** power
    o = verify(gpu_lib, c, [par])[0, 0]
    want, _, _ = ref_run(c, 0, slice(0, T), par, c["state"][0, 0], 1e-6, 128 ** -0.5)
    rows_close(o, want)


@pytest.mark.parametrize("what", ["row", "feature"])
@pytest.mark.parametrize("power", [10, 16, 19, 22, 24, 26, 28, 31, 60, 100])
@pytest.mark.parametrize("n, j", [(24, 20), (64, 63), (150, 40), (150, 64), (150, 149)])
def test_a_large_value_reaches_later_tokens_only(gpu_lib, n, j, power, what):
    """One token's v 2^power times the others': earlier tokens are as exact as without it, the state relative to its rows."""
    for fresh in (False, True):
        c = case(n + power, 1, 2, (2 * n,), 1, 3, 128, 128)
        if fresh:
            c["state"].zero_()
        want, S, MW = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 1e-6, 128 ** -0.5)
        enlarge(c["v"][0, j], power, what)
        out = torch.empty_like(c["state"])
        o, _ = scan(gpu_lib, c, [0, n, 2 * n], n, out)
        close_o(o[0, :j], want[:j], MW, n, 128, 128 ** -0.5)
        rows_close(o[0, :j], want[:j])
        if what == "feature":
            rows_close(o[0, :j, -1, 37].unsqueeze(0), want[:j, -1, 37].unsqueeze(0))
            others = [f for f in range(128) if f != 37]
            close_o(o[0, :n][..., others], want[..., others], MW, n, 128, 128 ** -0.5)
            close_state(out[0, 0][:, others], S[-1][:, others], MW, n, 128)
        # what sees it is as exact as the largest values it is summed from
        want, S, MW = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 1e-6, 128 ** -0.5)
        within_o(o[0, j:n], want[j:], MW, n, 128, 128 ** -0.5)
        within_state(out[0, 0], S[-1], MW, n, 128)
        want, S, MW = ref_run(c, 0, slice(n, 2 * n), list(range(-1, n - 1)), c["state"][0, 1], 1e-6, 128 ** -0.5)
        close_o(o[0, n:], want, MW, n, 128, 128 ** -0.5)
        close_state(out[0, 1], S[-1], MW, n, 128)


@pytest.mark.parametrize("power", [-10, -20, -24, -26, -30, -40, -90])
@pytest.mark.parametrize("n", [30, 64, 130])
def test_small_first_tokens_before_larger_ones(gpu_lib, n, power):
    c = case(n, 1, 1, (n,), 1, 2, 128, 128)
    c["state"].zero_()
    c["v"][0, :3] *= 2.0 ** power
    out = torch.empty_like(c["state"])
    o, _ = scan(gpu_lib, c, [0, n], n, out)
    want, S, _ = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 1e-6, 128 ** -0.5)
    rows_close(o[0], want)
    rows_close(out[0, 0], S[-1], 2.0 ** -18)


@pytest.mark.parametrize("power", [0, 7, 10, 14, 20, 40, 90])
@pytest.mark.parametrize("g", [-float("inf"), -45.0, -20.0, -16.0, -11.0])
@pytest.mark.parametrize("T, j", [(3, 0), (16, 0), (40, 0), (64, 0), (16, 3), (64, 9)])
def test_a_forgotten_state_leaves_the_tree_exact(gpu_lib, T, j, g, power):
    """Node j forgets a state 2^power times its usual size: what j and its descendants give is as exact as from the state
    that is left (e^g of it), however large the forgotten one was."""
    par = tree(np.random.default_rng(T + j), T, "random")
    below = [i for i in range(T) if j in _path(par, i)]
    c = case(T + power, 1, 1, (1, T), 1, 2, 128, 128)
    c["state"] *= 2.0 ** power
    c["g"][0, 0, j] = g
    o = verify(gpu_lib, c, [par])[0, 0]
    want, states, MW = ref_run(c, 0, slice(0, T), par, c["state"][0, 0], 1e-6, 128 ** -0.5)
    within_o(o, want, MW, T, 128, 128 ** -0.5)
    # the same nodes from the state that j leaves behind: their own magnitudes, not those of what was forgotten
    before = c["state"][0, 0].double() if j == 0 else states[par[j]]
    part = {x: c[x][:, 0, below] for x in ("q", "k", "v", "g", "beta")}
    part["g"] = part["g"].clone()
    part["g"][0, 0] = 0.0
    sub = [below.index(par[i]) if i != j else -1 for i in below]
    want2, _, MW = ref_run(part, 0, slice(0, len(below)), sub, torch.exp(torch.tensor(g, dtype=torch.float64, device=DEV)) * before, 1e-6, 128 ** -0.5)
    assert (want2 - want[below]).norm() <= 1e-9 * want2.norm()
    close_o(o[below], want[below], MW, T, 128, 128 ** -0.5)


@pytest.mark.parametrize("what", ["state", "tokens"])
@pytest.mark.parametrize("power", [0, 7, 10, 14, 20, 40, 90])
@pytest.mark.parametrize("g", [-float("inf"), -45.0, -20.0, -16.0, -11.0])
@pytest.mark.parametrize("n, j", [(24, 0), (24, 11), (64, 63), (150, 0), (150, 64), (150, 100)])
def test_a_forgotten_state_leaves_the_scan_exact(gpu_lib, n, j, g, power, what):
    """Token j forgets a state, or the writes of the tokens before it, 2^power times the usual size: o and the state from j on
    are as exact as from what is left of it."""
    c = case(n + power, 1, 1, (n,), 1, 2, 128, 128)
    if what == "state":
        c["state"] *= 2.0 ** power
    else:
        c["v"][0, :j] *= 2.0 ** power
    c["g"][0, j] = g
    out = torch.empty_like(c["state"])
    o, _ = scan(gpu_lib, c, [0, n], n, out)
    want, states, MW = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 1e-6, 128 ** -0.5)
    within_o(o[0], want, MW, n, 128, 128 ** -0.5)
    before = c["state"][0, 0].double() if j == 0 else states[j - 1]
    part = {x: c[x][:, j:] for x in ("q", "k", "v", "g", "beta")}
    part["g"] = part["g"].clone()
    part["g"][0, 0] = 0.0
    m = n - j
    want, S, MW = ref_run(part, 0, slice(0, m), list(range(-1, m - 1)), torch.exp(torch.tensor(g, dtype=torch.float64, device=DEV)) * before,
                          1e-6, 128 ** -0.5)
    assert (S[-1] - states[-1]).norm() <= 1e-9 * S[-1].norm()
    # beside the products' errors of close_o and close_state: the weight of an earlier write of the same block is held
    # down to 2^-37, once in the matrix and once in its inverse (P: 2^-33), so 64 of them leave at most
    M0, W0 = MW
    big = 0.0 if g == -float("inf") else 64 * c["v"][0, :j].double().abs().max().item() if j else 0.0
    close_o(o[0, j:], want, (M0 + 2.0 ** 12 * 2.0 ** -33 * big, W0), n, 128, 128 ** -0.5)
    err = (out[0, 0].double() - S[-1]).abs().max().item()
    assert err <= n * ((128 / 8 + 8) * 2.0 ** -24 * M0 + 2.0 ** -22 * M0 + 2.0 ** -21 * W0) + 2.0 ** -36 * big
    if g == -float("inf") or what == "state":
        close_state(out[0, 0], S[-1], MW, n, 128)


@pytest.mark.parametrize("n", [30, 64, 150])
def test_a_state_that_only_decays(gpu_lib, n):
    """Without writes (beta 0, or v and the state's product with k 0) the state is its decayed self, also where the decay of a
    block passes what fp16 holds; after large writes that are forgotten, small ones are not lost."""
    c = case(n, 1, 1, (n,), 1, 2, 128, 128)
    c["beta"].zero_()
    c["g"][:] = -0.9
    out = torch.empty_like(c["state"])
    scan(gpu_lib, c, [0, n], n, out)
    want = c["state"].double() * torch.exp(c["g"].double().sum(1))[:, None, :, None, None]
    assert ((out.double() - want).abs() <= n * 2.0 ** -22 * want.abs() + 1e-40).all()  # a rounding and an exp (2 ulp) per token
    c = case(n, 1, 1, (n,), 1, 2, 128, 128)  # writes, then none while what was written decays by e^-27
    c["beta"][0, n - 30:] = 0.0
    c["g"][0, n - 30:] = -0.9
    scan(gpu_lib, c, [0, n], n, out)
    _, S, _ = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 1e-6, 1.0)
    assert (out[0, 0].double() - S[-1]).norm() <= 2.0 ** -18 * S[-1].norm()


@pytest.mark.parametrize("log_s, g", [(120, -84.0), (124, -88.0), (126, -87.5), (40, -20.0), (-100, 0.0)])
def test_a_state_at_the_ends_of_fp32(gpu_lib, log_s, g):
    """A state near fp32's largest that a first decay brings to ordinary size, and one near its smallest."""
    rng = np.random.default_rng(5)
    for T in (3, 64):
        c = case(T, 1, 1, (1, T), 1, 2, 128, 128)
        c["state"] = torch.sign(c["state"]) * 2.0 ** (log_s - 1) * (1 + torch.rand_like(c["state"]))
        c["g"][0, 0, 0] = g
        par = tree(rng, T, "random")
        o = verify(gpu_lib, c, [par])[0, 0]
        want, _, _ = ref_run(c, 0, slice(0, T), par, c["state"][0, 0], 1e-6, 128 ** -0.5)
        after = {x: c[x].clone() for x in c}
        after["g"][0, 0, 0] = 0.0
        left = c["state"][0, 0].double() * np.exp(g)
        _, _, MW = ref_run(after, 0, slice(0, T), par, left, 1e-6, 128 ** -0.5)
        close_o(o, want, MW, T, 128, 128 ** -0.5)
    n = 100
    c = case(n, 1, 1, (n,), 1, 2, 128, 128)
    c["state"] = torch.sign(c["state"]) * 2.0 ** (log_s - 1) * (1 + torch.rand_like(c["state"]))
    c["g"][0, 0] = g
    out = torch.empty_like(c["state"])
    o, _ = scan(gpu_lib, c, [0, n], n, out)
    want, S, _ = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0], 1e-6, 128 ** -0.5)
    c["g"][0, 0] = 0.0
    _, _, MW = ref_run(c, 0, slice(0, n), list(range(-1, n - 1)), c["state"][0, 0].double() * np.exp(g), 1e-6, 128 ** -0.5)
    close_o(o[0], want, MW, n, 128, 128 ** -0.5)
    close_state(out[0, 0], S[-1], MW, n, 128)
