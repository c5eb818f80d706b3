"""What follows a target's layers, in 8 bits: the last norm, products with 8-bit weights, log probabilities.

Four operators that a verify round, or a decoding step, runs one after the other:

  norm      the residual's addition and the root-mean-square norm, with the sum, the normed rows and the normed rows in
            8 bits (e4m3 codes, one fp32 scale per 128 features of a row)
  matmul    rows in 8 bits times weights in 8 bits (e4m3, one fp32 scale per block of 128 x 128)
  head      the LM head with such weights: bf16 rows in, each row's largest logit and its token out
  logprobs  of a row of logits: the log probability and the rank of a given token, the entropy, the likeliest tokens
            with their log probabilities

The sizes are those of this repository's workloads (hidden 5120, 24 query heads of 256, a vocabulary of 248320; trees of
3, 16 and 64 nodes; prompts of 16391 tokens) and generic ones beside them (an inner size of 4 x 5120, odd rows and columns).

Formulas, for one row:
    norm      h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight
    8 bits    per 128 features: scale = max |y| / 448, code = e4m3(y / scale); a group of zeros has scale 0 and codes 0
    matmul    out[m, n] = sum over k of a[m, k] a_scale[m, k // 128] w[n, k] w_scale[n // 128, k // 128]
    logprobs  z = logits / temperature;  logp(t) = z_t - log sum exp z;  entropy = - sum p log p;  rank(t) = how many
              tokens have a larger logit, or the same one and a lower index
"""
import math
import random

import torch

own = False

EPS = 1e-6
BLOCK = 128  # features per scale of a row, rows and features per scale of a weight
TOP = 448.0  # the largest e4m3 value
TYPES = dict(bf16=torch.bfloat16, f16=torch.float16, f32=torch.float32)


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # one user's token through the last norm: latency counts
        dict(name="norm_token", op="norm", rows=1, H=5120, dtype="bf16", residual=True, wide=True, codes=True),
        # a served batch's 64-node trees, on the way into 8-bit weights only
        dict(name="norm_tree64_b32", op="norm", rows=2048, H=5120, dtype="bf16", residual=True, wide=False, codes=True),
        # a long prompt of odd length, plain 16-bit output
        dict(name="norm_prompt", op="norm", rows=16391, H=5120, dtype="bf16", residual=True, wide=True, codes=False),
        # rows whose length is no multiple of anything, in fp16, without a residual
        dict(name="norm_odd", op="norm", rows=515, H=2573, dtype="f16", residual=False, wide=True, codes=True),
        # one token's query projection, and the output projection of a 64-node tree: weights are read once
        dict(name="matmul_token", op="matmul", rows=1, K=5120, N=6144, out="bf16"),
        dict(name="matmul_tree64", op="matmul", rows=64, K=6144, N=5120, out="bf16"),
        # a prompt's widest product
        dict(name="matmul_prompt", op="matmul", rows=8199, K=5120, N=20480, out="bf16"),
        # small odd sizes, fp32 out
        dict(name="matmul_odd", op="matmul", rows=333, K=1040, N=1001, out="f32"),
        # one user's chain of three nodes through the LM head, and a served batch's 64-node trees
        dict(name="head_chain3", op="head", rows=3, H=5120, V=248320),
        dict(name="head_tree64_b32", op="head", rows=2048, H=5120, V=248320),
        # the sampled tokens of one user's chain, and of a served batch's trees with twenty alternatives each
        dict(name="logprobs_chain3", op="logprobs", rows=3, V=248320, dtype="f32", top=5, masked=0.0, t=1.0),
        dict(name="logprobs_tree64_b32", op="logprobs", rows=2048, V=248320, dtype="f32", top=20, masked=0.02, t=1.0),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "matmul", "head", "logprobs", "logprobs"])
    if op == "norm":
        c = dict(op=op, rows=_log(rng, 1, 16391), H=_log(rng, 64, 20480), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                 residual=rng.random() < 0.7, wide=rng.random() < 0.6)
        c["codes"] = not c["wide"] or rng.random() < 0.6
        if rng.random() < 0.6:
            c["H"] = -(-c["H"] // 64) * 64
        c["rows"] = min(c["rows"], 16391 * 5120 // c["H"])
        return c
    if op == "matmul":
        c = dict(op=op, rows=_log(rng, 1, 8199), K=16 * _log(rng, 4, 1280), N=_log(rng, 16, 20480),
                 out=rng.choice(["bf16", "bf16", "f16", "f32"]))
        if rng.random() < 0.6:
            c["K"], c["N"] = -(-c["K"] // 128) * 128, -(-c["N"] // 64) * 64
        while c["rows"] * c["K"] * c["N"] > 8199 * 5120 * 20480:
            c["rows"] = c["rows"] * 3 // 4
        return c
    if op == "head":
        c = dict(op=op, rows=_log(rng, 1, 2048), H=16 * _log(rng, 16, 512), V=_log(rng, 1000, 248320))
        while c["H"] * c["V"] > 5120 * 248320:
            c["H"] -= 16
        return c
    return dict(op=op, rows=_log(rng, 1, 2048), V=_log(rng, 100, 248320), dtype=rng.choice(["f32", "f32", "bf16", "f16"]),
                top=rng.choice([0, 1, 5, 20, 64, rng.randint(1, 64)]), masked=rng.choice([0.0, 0.0, 0.02, 0.9]),
                t=rng.choice([1.0, 1.0, 0.7, 1.3]))


# ----------------------------------------------------------------------------- inputs
def _blocks(n):
    return -(-n // BLOCK)


def _weights(n, k, gen, dev):
    """e4m3 weights [n, k] with one scale per block of 128 x 128, as an 8-bit checkpoint has them."""
    codes = torch.empty(n, k, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(_blocks(n), _blocks(k), device=dev)
    for i in range(0, n, 16384):  # a part at a time: 5 GB in 32 bits otherwise
        m = min(16384, n - i)
        w = torch.zeros(_blocks(m) * BLOCK, _blocks(k) * BLOCK, device=dev)
        w[:m, :k] = 0.02 * torch.randn(m, k, generator=gen, device=dev)
        w = w.view(_blocks(m), BLOCK, _blocks(k), BLOCK)
        s = w.abs().amax((1, 3)) / TOP
        codes[i:i + m] = (w / s[:, None, :, None]).reshape(_blocks(m) * BLOCK, -1)[:m, :k].to(torch.float8_e4m3fn)
        scale[i // BLOCK:i // BLOCK + _blocks(m)] = s
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    n = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    op, rows = case["op"], case["rows"]
    s = dict(case=case)
    if op == "norm":
        H, dt = case["H"], TYPES[case["dtype"]]
        loud = 1 + 30 * (torch.rand(H, generator=gen, device=dev) < 0.004)  # a few features are far louder than the rest
        s.update(x=(n(rows, H) * loud).to(dt), weight=(1 + 0.2 * n(H)).to(dt))
        if case["residual"]:
            s.update(residual=(4 * n(rows, H) * loud).to(dt), residual_out=torch.empty(rows, H, dtype=dt, device=dev))
        if case["wide"]:
            s["out"] = torch.empty(rows, H, dtype=dt, device=dev)
        if case["codes"]:
            s["out8"] = torch.empty(rows, H, dtype=torch.float8_e4m3fn, device=dev)
            s["out8_scale"] = torch.empty(rows, _blocks(H), device=dev)
    elif op == "matmul":
        K, N = case["K"], case["N"]
        s["a"], s["a_scale"] = _codes(n(rows, K))
        s["w"], s["w_scale"] = _weights(N, K, gen, dev)
        s["out"] = torch.empty(rows, N, dtype=TYPES[case["out"]], device=dev)
    elif op == "head":
        H, V = case["H"], case["V"]
        s["w"], s["w_scale"] = _weights(V, H, gen, dev)
        # rows that point at a token, as a trained model's do
        token = torch.randint(0, V, (rows,), generator=gen, device=dev)
        toward = s["w"][token].float() * s["w_scale"][token // BLOCK].repeat_interleave(BLOCK, dim=1)[:, :H]
        s["hidden"] = (n(rows, H) + 14 / math.sqrt(H) * toward / 0.02).bfloat16()
        s.update(argmax=torch.empty(rows, dtype=torch.int32, device=dev), maxlogit=torch.empty(rows, device=dev))
    else:
        V = case["V"]
        z = 2.5 * n(rows, V)
        z += 6 * (torch.rand(rows, 1, generator=gen, device=dev) * n(rows, V).clamp(min=3.2).sub_(3.2))  # a few likely tokens
        token = torch.randint(0, V, (rows,), generator=gen, device=dev)
        best = z.argmax(1)
        token = torch.where(torch.rand(rows, generator=gen, device=dev) < 0.6, best, token)  # most drawn tokens are likely ones
        if case["masked"]:
            hidden = torch.rand(rows, V, generator=gen, device=dev) < case["masked"]
            hidden[torch.arange(rows, device=dev), token] = False
            z.masked_fill_(hidden, float("-inf"))  # tokens that a grammar or a filter rules out
        s.update(logits=z.to(TYPES[case["dtype"]]), targets=token.int(), logp=torch.empty(rows, device=dev),
                 entropy=torch.empty(rows, device=dev), rank=torch.empty(rows, dtype=torch.int32, device=dev))
        if case["top"]:
            k = case["top"]
            s.update(top_tokens=torch.empty(rows, k, dtype=torch.int32, device=dev), top_logp=torch.empty(rows, k, device=dev))
    if own and op in ("head", "logprobs"):
        import tree_speculative_decoding_array_gb300 as tsv

        size = (tsv.lm_head_workspace_size(rows, case["H"], case["V"], tsv.E4M3_B128) if op == "head"
                else tsv.token_logprobs_workspace_size(rows, case["V"], case["top"]))
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device=dev)
    return s


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import tree_speculative_decoding_array_gb300 as tsv

        if c["op"] == "norm":
            tsv.add_rms_norm(s["x"], s["weight"], eps=EPS, residual=s.get("residual"), residual_out=s.get("residual_out"),
                             out=s.get("out"), out8=s.get("out8"), out8_scale=s.get("out8_scale"))
            return {k: s[k] for k in ("residual_out", "out", "out8", "out8_scale") if k in s}
        if c["op"] == "matmul":
            tsv.matmul_e4m3(s["a"], s["a_scale"], s["w"], s["w_scale"], s["out"])
            return s["out"]
        if c["op"] == "head":
            tsv.lm_head_argmax(s["hidden"], s["w"], s["argmax"], w_dtype=tsv.E4M3_B128, V=c["V"], scales=s["w_scale"],
                               maxlogit=s["maxlogit"], workspace=s["workspace"])
            return s["argmax"], s["maxlogit"]
        tsv.token_logprobs(s["logits"], s["targets"], s["logp"], rank=s["rank"], entropy=s["entropy"], temperature=c["t"],
                           top_tokens=s.get("top_tokens"), top_logp=s.get("top_logp"), workspace=s["workspace"])
        return {k: s[k] for k in ("logp", "entropy", "rank", "top_tokens", "top_logp") if k in s}
    return dict(norm=_norm, matmul=_matmul, head=_head, logprobs=_logprobs)[c["op"]](s)


def _codes(y):
    """Rows in 8 bits: e4m3 codes and the scale of every 128 features."""
    H = y.shape[1]
    g = torch.nn.functional.pad(y, (0, _blocks(H) * BLOCK - H)).view(y.shape[0], _blocks(H), BLOCK)
    scale = g.abs().amax(-1) / TOP
    q = torch.where(scale[..., None] > 0, g / scale[..., None], torch.zeros((), device=y.device))
    return q.flatten(1)[:, :H].to(torch.float8_e4m3fn), scale


def _values(codes, scale, rows_per_scale):
    """fp32 values of e4m3 codes [n, k] with a scale per `rows_per_scale` rows and 128 features."""
    s = scale.repeat_interleave(rows_per_scale, dim=0)[:codes.shape[0]]
    return codes.float() * s.repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]


def _norm(s):
    h = s["x"].float()
    got = {}
    if "residual" in s:
        h = h + s["residual"].float()
        got["residual_out"] = h.to(s["x"].dtype)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if "out" in s:
        got["out"] = y.to(s["x"].dtype)
    if "out8" in s:
        got["out8"], got["out8_scale"] = _codes(y)
    return got


def _matmul(s):
    return torch.matmul(_values(s["a"], s["a_scale"], 1), _values(s["w"], s["w_scale"], BLOCK).T).to(s["out"].dtype)


def _head(s):
    a = _values(*_codes(s["hidden"].float()), 1)
    logits = torch.matmul(a, _values(s["w"], s["w_scale"], BLOCK).T)
    best = logits.amax(-1)
    token = torch.arange(logits.shape[1], device=logits.device)
    return torch.where(logits == best[:, None], token, logits.shape[1]).amin(-1).int(), best


def _logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    z = x / c["t"]
    z = z - z.amax(-1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(-1, keepdim=True)
    mean = torch.where(e > 0, e * z, torch.zeros((), device=z.device)).sum(-1, keepdim=True) / total
    z -= torch.log(total)
    at = s["targets"].long()[:, None]
    t = x.gather(1, at)
    token = torch.arange(c["V"], device=x.device)
    got = dict(logp=z.gather(1, at)[:, 0], entropy=(torch.log(total) - mean)[:, 0],
               rank=((x > t) | ((x == t) & (token < at))).sum(-1).int())
    if c["top"]:
        best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        got.update(top_tokens=best.int(), top_logp=z.gather(1, best))
    return got


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, rows = case["op"], case["rows"]
    if op == "norm":
        H, elt = case["H"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": rows * (H * elt * (1 + 2 * case["residual"] + case["wide"]) + case["codes"] * (H + 4 * _blocks(H))) + H * elt,
                "flops": 6.0 * rows * H}
    if op == "matmul":
        K, N = case["K"], case["N"]
        return {"bytes": (rows + N) * K + 4 * _blocks(K) * (rows + _blocks(N)) + rows * N * (4 if case["out"] == "f32" else 2),
                "flops": 2.0 * rows * K * N}
    if op == "head":
        H, V = case["H"], case["V"]
        return {"bytes": rows * (2 * H + 8) + V * H + 4 * _blocks(H) * _blocks(V), "flops": 2.0 * rows * H * V}
    return {"bytes": rows * (case["V"] * (4 if case["dtype"] == "f32" else 2) + 16 + 8 * case["top"]), "flops": 6.0 * rows * case["V"]}


# ----------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, rows = case["op"], case["rows"]
    if op == "norm":
        H = case["H"]
        h = s["x"].double()
        got = {}
        if case["residual"]:
            h = got["residual_out"] = h + s["residual"].double()
        y = h * (h.square().sum(1) / H + EPS).rsqrt().unsqueeze(1) * s["weight"].double()
        if case["wide"]:
            got["out"] = y
        if case["codes"]:
            got["out8"], got["out8_scale"] = torch.empty_like(y), torch.empty(rows, _blocks(H), dtype=torch.float64, device=y.device)
            for j in range(_blocks(H)):
                part = y[:, j * BLOCK:(j + 1) * BLOCK]
                got["out8_scale"][:, j] = part.abs().max(1).values / TOP
                got["out8"][:, j * BLOCK:(j + 1) * BLOCK] = part / got["out8_scale"][:, j:j + 1]
        return got
    if op == "matmul":
        return _product(s["a"], s["a_scale"], s["w"], s["w_scale"], 0, case["N"])
    if op == "head":
        # the rows' codes are whole decisions, so they are taken as the definition takes them: in 32 bits
        a, a_scale = _codes(s["hidden"].float())
        best, at = torch.full((rows,), -math.inf, dtype=torch.float64, device=a.device), None
        at = torch.zeros(rows, dtype=torch.int64, device=a.device)
        for i in range(0, case["V"], 16384):
            m, j = _product(a, a_scale, s["w"], s["w_scale"], i, min(case["V"], i + 16384)).max(1)
            at = torch.where(m > best, j + i, at)
            best = torch.maximum(m, best)
        return at.int(), best
    logp, entropy, rank, tokens, top = [], [], [], [], []
    for i in range(0, rows, 128):
        x = s["logits"][i:i + 128].double()
        lp = torch.log_softmax(x / case["t"], dim=1)
        at = s["targets"][i:i + 128].long()
        r = torch.arange(x.shape[0], device=x.device)
        logp.append(lp[r, at])
        entropy.append(torch.special.entr(lp.exp()).sum(1))
        better = x > x[r, at].unsqueeze(1)
        same_before = (x == x[r, at].unsqueeze(1)).cumsum(1)[r, at] - 1
        rank.append(better.sum(1) + same_before)
        if case["top"]:
            top.append(lp.topk(case["top"], dim=1).values)
    got = dict(logp=torch.cat(logp), entropy=torch.cat(entropy), rank=torch.cat(rank).int())
    if case["top"]:
        got.update(top_tokens=None, top_logp=torch.cat(top))  # whole values: the plain form's have to be met
    return got


def _product(a, a_scale, w, w_scale, lo, hi):
    """Rows lo .. hi of the weights (lo a multiple of 128), block of features by block of features."""
    out = torch.zeros(a.shape[0], hi - lo, dtype=torch.float64, device=a.device)
    for j in range(_blocks(a.shape[1])):
        f = slice(j * BLOCK, (j + 1) * BLOCK)
        part = a[:, f].double() @ w[lo:hi, f].double().t()
        per_row = w_scale[lo // BLOCK:, j].double().repeat_interleave(BLOCK)[:hi - lo]
        out += part * a_scale[:, j:j + 1].double() * per_row
    return out
