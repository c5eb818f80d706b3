"""The operators of a hybrid target's layers in a verify round, as cases that can be measured.

A hybrid target alternates layers of the gated delta rule (a matrix-valued recurrent state per head) with
full-attention layers.  Four operators:

  verify   every node of a draft tree through the recurrent layers, each from its own parent's state
  commit   the recurrent states advanced along the accepted path
  scan     the states advanced over new tokens: single tokens, prompts, ragged batches of them
  attend   the block's attention over a cache held in 4 bits (affine, groups of 64 features)

The sizes are those of this repository's workloads (16 full-attention layers with 24 query and 4 KV heads of 256;
trees of 3, 16 and 64 nodes) with 48 recurrent layers beside them, 16 key and 48 value heads of 128.

Gated delta rule, for one value head with state S [DV, DK], log decay g <= 0 and write strength beta:
    S <- e^g S;  u = beta (v - S k);  S <- S + u k^T;  o = S q / sqrt(DK)
q and k are divided by their norms first: x / sqrt(sum x^2 + 1e-6).  Value head h reads key head h // (HV / HK).
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
CHUNK = 64  # tokens per block of the scan's plain form
GROUP = 64  # features per scale and bias of a 4-bit row


# ----------------------------------------------------------------------------- the cases
def listed():
    hyb = dict(HK=16, HV=48, D=128)
    att = dict(HQ=24, HKV=4, D=256)
    return [
        # one user's chain of three drafted tokens through every recurrent layer: latency counts
        dict(name="verify_chain3", op="verify", L=48, B=1, T=3, depth=2, tree=1, **hyb),
        # one user's 16-node tree
        dict(name="verify_tree16", op="verify", L=48, B=1, T=16, depth=5, tree=2, **hyb),
        # a served batch with 64-node trees
        dict(name="verify_tree64_b32", op="verify", L=48, B=32, T=64, depth=8, tree=3, **hyb),
        # the round's end for one user and for the served batch
        dict(name="commit_tree16", op="commit", L=48, B=1, T=16, most=6, path=4, **hyb),
        dict(name="commit_tree64_b32", op="commit", L=48, B=32, T=64, most=9, path=5, **hyb),
        # plain decoding, one layer's call: one user's token, and a batch's
        dict(name="scan_token", op="scan", L=1, B=1, least=1, most=1, lens=6, **hyb),
        dict(name="scan_token_b64", op="scan", L=1, B=64, least=1, most=1, lens=7, **hyb),
        # one layer's call over one long prompt of odd length, and over a batch of prompts from short to long
        dict(name="scan_prompt", op="scan", L=1, B=1, least=16391, most=16391, lens=8, **hyb),
        dict(name="scan_ragged_b24", op="scan", L=1, B=24, least=5, most=4001, lens=9, **hyb),
        # single tokens of a batch over long 4-bit caches of several lengths
        dict(name="attend_token_b32", op="attend", L=4, B=32, T=1, S=32768, ragged=True, depth=0, tree=10, **att),
        # one user's 16-node tree over every full-attention layer
        dict(name="attend_tree16", op="attend", L=16, B=1, T=16, S=8192, ragged=False, depth=5, tree=11, **att),
        # a served batch with 64-node trees
        dict(name="attend_tree64_b8", op="attend", L=4, B=8, T=64, S=32768, ragged=True, depth=8, tree=12, **att),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["verify", "commit", "scan", "scan", "attend"])
    seed = rng.randrange(1 << 30)
    if op == "attend":
        HKV = rng.choice([1, 2, 4, 8])
        c = dict(op=op, L=_log(rng, 1, 16), HKV=HKV, HQ=HKV * rng.choice([1, 2, 4, 6, 8]), D=rng.choice([128, 256, 256]),
                 T=_log(rng, 1, 64), B=_log(rng, 1, 32), S=_log(rng, 1, 40000), ragged=rng.random() < 0.7, tree=seed)
        c["depth"] = rng.randint(0 if c["T"] == 1 else 1, max(1, min(c["T"] - 1, 12))) if c["T"] > 1 else 0
        while c["L"] * c["B"] * HKV * c["S"] > 2 ** 21 or c["L"] * c["B"] * c["HQ"] * c["T"] * c["S"] > 2 ** 30:
            if c["S"] > 4096:
                c["S"] = c["S"] * 3 // 4 + 1
            else:
                c["L"], c["B"] = max(1, c["L"] // 2), max(1, c["B"] * 3 // 4)
        return c
    HK = rng.choice([4, 8, 16])
    c = dict(op=op, HK=HK, HV=HK * rng.choice([1, 2, 3, 4] if HK < 16 else [1, 2, 3]), D=128)
    if op == "scan":
        c["L"], c["B"] = 1, _log(rng, 1, 64)
        if rng.random() < 0.4:
            c["least"] = 1
            c["most"] = rng.choice([1, 1, rng.randint(2, 8)])
        else:
            c["most"] = _log(rng, 9, 16391)
            c["least"] = rng.randint(0, c["most"])
            while c["B"] > 1 and c["B"] * c["most"] > 40000:
                c["B"] = c["B"] // 2
        c["lens"] = seed
        return c
    c["L"], c["B"], c["T"] = _log(rng, 1, 48), _log(rng, 1, 32), _log(rng, 1, 64)
    if op == "verify":
        c["depth"] = rng.randint(1, min(c["T"] - 1, 12)) if c["T"] > 1 else 0
        c["tree"] = seed
    else:
        c["most"] = rng.randint(1, min(c["T"], 12))
        c["path"] = seed
    return c


def _lens(case):
    """New tokens of each sequence of a scan (the longest is `most`)."""
    r = random.Random(case["lens"])
    lo, hi = math.log(case["least"] + 1), math.log(case["most"] + 1)
    n = [min(case["most"], int(round(math.exp(r.uniform(lo, hi)))) - 1) for _ in range(case["B"])]
    n[r.randrange(case["B"])] = case["most"]
    return [max(case["least"], x) for x in n]


def _history(case):
    """Cached positions ahead of the block, per sequence (the longest is S)."""
    r = random.Random(case["tree"] + 1)
    n = [r.randint(max(1, case["S"] // 2), case["S"]) if case["ragged"] else case["S"] for _ in range(case["B"])]
    n[0] = case["S"]
    return n


def _paths(case):
    """Accepted paths: strictly increasing node lists that start at the root."""
    r = random.Random(case["path"])
    out = []
    for b in range(case["B"]):
        n = case["most"] if b == 0 else r.randint(1, case["most"])
        out.append([0] + sorted(r.sample(range(1, case["T"]), n - 1)))
    return out


def _parents(case):
    """A random topological tree per sequence, of the case's depth."""
    r = random.Random(case["tree"])
    rows = []
    for _ in range(case["B"]):
        par, dep = [-1], [0]
        for i in range(1, case["T"]):
            p = i - 1 if i <= case["depth"] else r.choice([j for j in range(i) if dep[j] < case["depth"]])
            par.append(p)
            dep.append(dep[p] + 1)
        rows.append(par)
    return rows


def _ancestors(parents):
    """bool [B, T, T]: [b, i, j] set where j is an ancestor of i or i itself; and the same as 64-bit words."""
    B, T = len(parents), len(parents[0])
    m = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for i, p in enumerate(parents[b]):
            if p >= 0:
                m[b, i] = m[b, p]
            m[b, i, i] = True
    words = (m.astype(np.uint64) << np.arange(T, dtype=np.uint64)).sum(axis=2, dtype=np.uint64)
    return m, words.view(np.int64)


# ----------------------------------------------------------------------------- inputs
def _recurrent_inputs(case, rows, gen, dev):
    """q, k, v rows, gates and states of every layer: rows is the shape ahead of the heads, [B, T] or [tokens]."""
    L, B, HK, HV, D = case["L"], case["B"], case["HK"], case["HV"], case["D"]
    n = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    # each head forgets at its own rate, from about 0.001 to 1.5 per token
    rate = torch.exp(u(L, HV) * 6.0 - 6.5).view(L, *[1] * len(rows), HV)
    return dict(
        q=n(L, *rows, HK, D).bfloat16(), k=n(L, *rows, HK, D).bfloat16(), v=n(L, *rows, HV, D).bfloat16(),
        g=-rate * (0.25 + 1.5 * u(L, *rows, HV)), beta=torch.sigmoid(n(L, *rows, HV)),
        state=0.2 * n(L, B, HV, D, D))


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    op, L, B = case["op"], case["L"], case["B"]
    s = dict(case=case)
    if op == "attend":
        T, HQ, HKV, D = case["T"], case["HQ"], case["HKV"], case["D"]
        hist = _history(case)
        cap = (max(hist) + T + 63) // 64 * 64
        mask, words = _ancestors(_parents(case))
        s.update(q=torch.randn(L, B, T, HQ, D, generator=gen, device=dev).bfloat16(), kv_len=i32([h + T for h in hist]),
                 anc=torch.from_numpy(words.copy()).to(dev), mask=torch.from_numpy(mask).to(dev), hist=hist,
                 status=torch.zeros(4, dtype=torch.int32, device=dev), o=torch.empty(L, B, T, HQ, D, dtype=torch.bfloat16, device=dev))
        for x in "kv":
            s[x] = torch.randint(0, 256, (L, B, HKV, cap, D // 2), generator=gen, device=dev, dtype=torch.uint8)
            sc = (0.25 + 0.15 * torch.rand(L, B, HKV, cap, D // GROUP, generator=gen, device=dev)).half()
            bi = (-7.5 * sc.float() + 0.1 * torch.randn(sc.shape, generator=gen, device=dev)).half()
            s[x + "_scale"] = torch.stack([sc, bi], dim=-1).contiguous()  # (scale, bias) of each group
    elif op == "scan":
        lens = _lens(case)
        s.update(_recurrent_inputs(case, (sum(lens),), gen, dev), lens=lens)
        s["cu_len"] = i32([0] + list(np.cumsum(lens)))
        s["state_out"], s["o"] = torch.empty_like(s["state"]), torch.empty_like(s["v"])
    else:
        s.update(_recurrent_inputs(case, (B, case["T"]), gen, dev), status=torch.zeros(4, dtype=torch.int32, device=dev))
        if op == "verify":
            parents = _parents(case)
            mask, words = _ancestors(parents)
            s.update(mask=torch.from_numpy(mask).to(dev), anc=torch.from_numpy(words.copy()).to(dev), o=torch.empty_like(s["v"]))
        else:
            paths = _paths(case)
            s.update(path=i32([p + [-1] * (case["T"] - len(p)) for p in paths]), path_len=i32([len(p) for p in paths]),
                     state_out=torch.empty_like(s["state"]))
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """What a serving program builds once over its buffers: the call's descriptor and workspace."""
    import tree_speculative_decoding_array_gb300 as tsv

    c, per = s["case"], lambda x: [s[x][l] for l in range(c["L"])]  # noqa: E731
    if c["op"] == "attend":
        d = tsv.attn_desc(per("q"), per("k"), per("v"), per("o"), s["kv_len"], s["anc"], T=c["T"], HQ=c["HQ"], HKV=c["HKV"],
                          D=c["D"], kv_dtype=tsv.I4_G64, max_kv_len=c["S"] + c["T"], k_scale=per("k_scale"), v_scale=per("v_scale"))
        return d, torch.empty(max(tsv.attention_workspace_size(d), 256), dtype=torch.uint8, device=s["q"].device)
    d = tsv.gdn_desc(per("q"), per("k"), per("v"), per("g"), per("beta"), per("state"),
                     o=per("o") if "o" in s else None, state_out=per("state_out") if "state_out" in s else None)
    return d, None


# ----------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import tree_speculative_decoding_array_gb300 as tsv

        d, ws = s["plan"]
        if op == "attend":
            tsv.tree_verify_attention(d, ws, dev_status=s["status"])
            return s["o"]
        if op == "verify":
            tsv.gdn_tree_verify(d, s["anc"], dev_status=s["status"])
            return s["o"]
        if op == "commit":
            tsv.gdn_commit(d, s["path"], s["path_len"], dev_status=s["status"])
            return s["state_out"]
        tsv.gdn_scan(d, s["cu_len"], max_len=s["case"]["most"])
        return s["o"], s["state_out"]
    return dict(attend=_attend, verify=_verify, commit=_commit, scan=_scan)[op](s)


def _unit(x):
    x = x.float()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def _heads(x, HV):
    """Key heads repeated for the value heads that read them: [..., HK, D] -> [..., HV, D]."""
    return x.repeat_interleave(HV // x.shape[-2], dim=-2)


def _verify(s):
    """The whole tree at once.  With G_i the decay summed from the root to node i, node i's write is
    u_i = beta_i (v_i - e^{G_i} S k_i - sum over strict ancestors j of e^{G_i - G_j} (k_j . k_i) u_j), a system that
    is triangular in the depth, so as many substitutions as the tree is deep solve it."""
    c = s["case"]
    B, T, HV, D, depth = c["B"], c["T"], c["HV"], c["D"], c["depth"]
    mask = s["mask"]
    strict = (mask & ~torch.eye(T, dtype=torch.bool, device=mask.device)).view(B, 1, T, T).float()
    seen = mask.view(B, 1, T, T).float()
    out = []
    for l in range(c["L"]):
        rows = lambda x: x.transpose(1, 2).contiguous()  # noqa: E731  [B, T, HV, D] -> [B, HV, T, D]
        q, k = rows(_heads(_unit(s["q"][l]), HV)) / math.sqrt(D), rows(_heads(_unit(s["k"][l]), HV))
        v, beta = rows(s["v"][l].float()), s["beta"][l].transpose(1, 2).unsqueeze(-1)
        G = torch.matmul(mask.double(), s["g"][l].double())  # [B, T, HV]: sums over ancestors and self
        G = G.transpose(1, 2)
        decay = torch.exp(((G.unsqueeze(-1) - G.unsqueeze(-2)) * seen).float()) * seen  # [B, HV, T, T]
        S = s["state"][l].transpose(-1, -2)  # [B, HV, DK, DV]
        e = torch.exp(G).float().unsqueeze(-1)
        A = beta * torch.matmul(k, k.transpose(-1, -2)) * decay * strict
        R = beta * (v - e * torch.matmul(k, S))
        U = R
        for _ in range(depth):
            U = R - torch.matmul(A, U)
        o = e * torch.matmul(q, S) + torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * decay, U)
        out.append(o.transpose(1, 2).bfloat16())
    return torch.stack(out)


def _commit(s):
    """One token of every sequence's path at a time; sequences whose path has ended keep their state."""
    c = s["case"]
    HV = c["HV"]
    S = s["state"]
    b = torch.arange(c["B"], device=S.device)
    for j in range(c["most"]):
        live = (s["path_len"] > j).view(1, -1, 1, 1, 1)
        i = s["path"][:, j].clamp(min=0).long()
        k, v = _heads(_unit(s["k"][:, b, i]), HV), s["v"][:, b, i].float()
        g, beta = s["g"][:, b, i], s["beta"][:, b, i]
        N = S * torch.exp(g)[..., None, None]
        u = beta[..., None] * (v - (N * k.unsqueeze(-2)).sum(-1))
        S = torch.where(live, N + u.unsqueeze(-1) * k.unsqueeze(-2), S)
    return S


def _scan(s):
    """Blocks of CHUNK tokens: inside a block the triangular system is inverted for all blocks at once, then the blocks
    are taken in order.  Sequences are padded to whole blocks with rows that neither write nor forget."""
    c = s["case"]
    B, HV, D, most = c["B"], c["HV"], c["D"], c["most"]
    C = min(CHUNK, most)
    n = (most + C - 1) // C
    dev = s["v"].device
    pos = torch.arange(n * C, device=dev).view(1, -1)
    length = (s["cu_len"][1:] - s["cu_len"][:-1]).long().view(-1, 1)
    real = pos < length  # [B, n * C]
    at = (s["cu_len"][:-1].long().view(-1, 1) + pos)[real]  # packed row of every real place
    outs, states = [], []
    for l in range(c["L"]):
        def spread(x):  # packed rows -> [B, HV, n, C, ...]
            y = torch.zeros(B, n * C, *x.shape[1:], dtype=torch.float32, device=dev)
            y[real] = x.float()[at]
            return y.view(B, n, C, *x.shape[1:]).movedim(3, 1)
        q, k = spread(_heads(_unit(s["q"][l]), HV)) / math.sqrt(D), spread(_heads(_unit(s["k"][l]), HV))
        v, beta = spread(s["v"][l]), spread(s["beta"][l]).unsqueeze(-1)
        G = spread(s["g"][l]).double().cumsum(-1)
        low = torch.tril(torch.ones(C, C, device=dev))
        decay = torch.exp(((G.unsqueeze(-1) - G.unsqueeze(-2)) * low).float()) * low
        A = beta * torch.matmul(k, k.transpose(-1, -2)) * decay * (1 - torch.eye(C, device=dev))
        inv = torch.eye(C, device=dev).expand_as(A)
        for _ in range(C - 1):
            inv = torch.eye(C, device=dev) - torch.matmul(A, inv)
        P = torch.matmul(q, k.transpose(-1, -2)) * decay
        e = torch.exp(G).float().unsqueeze(-1)
        rest = torch.exp(G[..., -1:] - G).float().unsqueeze(-1)
        S = s["state"][l].transpose(-1, -2)  # [B, HV, DK, DV]
        o = torch.empty_like(v)
        for j in range(n):
            ej = e[:, :, j]
            U = torch.matmul(inv[:, :, j], beta[:, :, j] * (v[:, :, j] - ej * torch.matmul(k[:, :, j], S)))
            o[:, :, j] = ej * torch.matmul(q[:, :, j], S) + torch.matmul(P[:, :, j], U)
            S = ej[:, :, -1:] * S + torch.matmul(k[:, :, j].transpose(-1, -2), rest[:, :, j] * U)
        rows = o.movedim(1, 3).reshape(B, n * C, HV, D)[real]
        outs.append(rows.bfloat16())
        states.append(S.transpose(-1, -2))
    return torch.stack(outs), torch.stack(states).contiguous()


def _values(codes, affine):
    """4-bit rows [..., D / 2] and their (scale, bias) [..., D / 64, 2] as the values they stand for; element 2j of a
    row is byte j's low nibble."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(affine.dtype)
    q = q.view(*q.shape[:-1], -1, GROUP)
    return (q * affine[..., :1] + affine[..., 1:]).flatten(-2)


def _attend(s):
    """Softmax attention of the block's rows over the whole history and their own ancestors, one sequence at a time."""
    c = s["case"]
    T, HKV, D = c["T"], c["HKV"], c["D"]
    G, dt = c["HQ"] // HKV, torch.float32
    o = torch.empty(c["L"], c["B"], T, c["HQ"], D, dtype=torch.bfloat16, device=s["q"].device)
    for b, S in enumerate(s["hist"]):
        hidden = ~s["mask"][b].repeat_interleave(G, dim=0)  # rows (node, head of the group)
        for l in range(c["L"]):
            K = _values(s["k"][l, b, :, :S + T], s["k_scale"][l, b, :, :S + T].to(dt))
            x = s["q"][l, b].to(dt).view(T, HKV, G, D).transpose(0, 1).reshape(HKV, T * G, D)
            x = torch.matmul(x, K.transpose(-1, -2)) / math.sqrt(D)
            x[:, :, S:].masked_fill_(hidden, float("-inf"))
            x = torch.exp(x - x.amax(-1, keepdim=True))
            x = x / x.sum(-1, keepdim=True)
            x = torch.matmul(x, _values(s["v"][l, b, :, :S + T], s["v_scale"][l, b, :, :S + T].to(dt)))
            o[l, b] = x.view(HKV, T, G, D).transpose(0, 1).reshape(T, c["HQ"], D)
    return o


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, L, B, D = case["op"], case["L"], case["B"], case["D"]
    if op == "attend":
        HQ, T = case["HQ"], case["T"]
        keys = sum(h + T for h in _history(case))
        return {"bytes": L * (case["HKV"] * keys * 2 * (D // 2 + 4 * (D // GROUP)) + 2 * B * T * HQ * D * 2 + B * T * 8 + B * 4),
                "flops": 4.0 * L * HQ * T * D * keys}
    HK, HV = case["HK"], case["HV"]
    state = L * B * HV * D * D * 4
    row = 2 * HK * D * 2 + HV * (D * 2 + 8)  # q, k, v and the two gates of a token
    if op == "verify":
        n = B * case["T"]
        # each node's two products with the state, its inner products with its ancestors and their writes
        return {"bytes": state + L * n * (row + HV * D * 2) + n * 8, "flops": 2.0 * L * n * HV * D * (2 * D + 4 * (case["depth"] + 1))}
    if op == "commit":
        n = sum(len(p) for p in _paths(case))
        return {"bytes": 2 * state + L * n * (row - HK * D * 2) + B * (case["T"] + 1) * 4, "flops": 5.0 * L * n * HV * D * D}
    n = sum(_lens(case))
    return {"bytes": 2 * state + L * n * (row + HV * D * 2) + (B + 1) * 4, "flops": 7.0 * L * n * HV * D * D}


# ----------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attend":
        return _attention_by_definition(s)
    unit = lambda x: x.double() / torch.sqrt(x.double().pow(2).sum(-1, keepdim=True) + EPS)  # noqa: E731
    HV, D = case["HV"], case["D"]
    L, B = case["L"], case["B"]

    def step(S, l, rows, want_o):
        """One token: S [B, HV, DV, DK] of layer l, `rows` picks each sequence's token out of the layer's inputs."""
        take = lambda x: torch.repeat_interleave(unit(x[l][rows]), HV // case["HK"], dim=1)  # noqa: E731
        k, v = take(s["k"]), s["v"][l][rows].double()
        S = S * torch.exp(s["g"][l][rows].double())[..., None, None]
        u = s["beta"][l][rows].double().unsqueeze(-1) * (v - torch.einsum("bhvk,bhk->bhv", S, k))
        S = S + torch.einsum("bhv,bhk->bhvk", u, k)
        return S, torch.einsum("bhvk,bhk->bhv", S, take(s["q"])) / math.sqrt(D) if want_o else None

    b = torch.arange(B, device=s["v"].device)
    if op == "verify":
        out = torch.empty(s["v"].shape, dtype=torch.float64, device=s["v"].device)
        parents = torch.tensor(_parents(case), device=b.device)
        for l in range(L):
            forks = torch.empty(case["T"], B, HV, D, D, dtype=torch.float64, device=b.device)
            for i in range(case["T"]):
                S = s["state"][l].double() if i == 0 else forks[parents[:, i], b]
                forks[i], out[l, :, i] = step(S, l, (b, torch.full_like(b, i)), True)
        return out
    if op == "commit":
        out = torch.empty(s["state"].shape, dtype=torch.float64, device=b.device)
        paths = _paths(case)
        for l in range(L):
            S = s["state"][l].double()
            for j in range(case["most"]):
                live = torch.tensor([n for n, p in enumerate(paths) if j < len(p)], device=b.device)
                node = torch.tensor([p[j] for p in paths if j < len(p)], device=b.device)
                S[live] = step(S[live], l, (live, node), False)[0]
            out[l] = S
        return out
    lens = s["lens"]
    if max(lens) > 20000:
        return None
    first = torch.tensor(np.cumsum([0] + lens[:-1]), device=b.device)
    o = torch.empty(s["v"].shape, dtype=torch.float64, device=b.device)
    out = torch.empty(s["state"].shape, dtype=torch.float64, device=b.device)
    by_length = sorted(range(B), key=lambda n: -lens[n])
    for l in range(L):
        S = s["state"][l].double()[by_length]  # the longest first, so that the live ones are a prefix
        live = B
        for t in range(max(lens)):
            while lens[by_length[live - 1]] <= t:
                live -= 1
            if t == 0 or live != seen:
                seen, rows = live, first[by_length[:live]]
            S[:live], o_t = step(S[:live], l, (rows + t,), True)
            o[l][rows + t] = o_t
        out[l][by_length] = S
    return o, out


def _attention_by_definition(s):
    c = s["case"]
    T, HQ, HKV, D = c["T"], c["HQ"], c["HKV"], c["D"]
    o = torch.empty(s["o"].shape, dtype=torch.float64, device=s["o"].device)

    def stored(x, l, b, h, n):
        """fp64 values of one head's first n rows."""
        byte = s[x][l, b, h, :n].to(torch.int64)
        code = torch.empty(n, D, dtype=torch.float64, device=byte.device)
        code[:, 0::2], code[:, 1::2] = (byte % 16).double(), torch.div(byte, 16, rounding_mode="floor").double()
        pair = s[x + "_scale"][l, b, h, :n].double()
        return code * pair[..., 0].repeat_interleave(GROUP, dim=1) + pair[..., 1].repeat_interleave(GROUP, dim=1)

    for b, S in enumerate(s["hist"]):
        allowed = torch.cat([torch.ones(T, S, dtype=torch.bool, device=o.device), s["mask"][b]], dim=1)
        for l in range(c["L"]):
            for h in range(HKV):
                heads = slice(h * (HQ // HKV), (h + 1) * (HQ // HKV))
                K, V = stored("k", l, b, h, S + T), stored("v", l, b, h, S + T)
                w = torch.einsum("thd,nd->thn", s["q"][l, b, :, heads].double(), K) * D ** -0.5
                w = torch.softmax(w.masked_fill(~allowed.unsqueeze(1), -math.inf), dim=-1)
                o[l, b, :, heads] = torch.einsum("thn,nd->thd", w, V)
    return o
