"""The norm with 8-bit output, 8-bit rows, products with 8-bit weights and the 8-bit LM head against the fp64 oracle.

Tolerances.  u = 2^-24 is half an fp32 step.
  norm      h: one addition (u) and one rounding.  y: a row's squares are added at most 64 in a row in a thread, then over
            lanes and warps (under 64 more), so the sum is off by 128 u, its root by half of that, and the quotient, root and products
            add 6 u: (64 + 6) u < 2^-17.  Below fp32's normal numbers each rounding is off by up to 2^-150 as it is: that of
            h / rms, which the weight then multiplies, and the last one; so (1 + |weight|) 2^-150.
  codes     of a y that is off by 2^-17: the scale is off by 2^-17 + u; a value is off by half a code's step (2^-4 of it, or
            2^-10 scales below the smallest normal code) and by the scale's error: bounded by 1 + 2^-13 of those.  A scale below
            fp32's normal numbers is off by up to 2^-150, 448 times of which the largest code is off by.
  matmul    products of two codes are exact in fp32.  128 of them are added in fp32 (at most a whole step, 2^-23, per addition
            where an addition truncates), scaled (2 u) and added over the blocks (u each), all relative to the sum of |terms|.
"""
import numpy as np
import pytest
import torch

from oracle import rows8

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the smallest subnormal
F8 = torch.float8_e4m3fn


def rnd(*shape, seed=0, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def bytes_of(t):
    return t.cpu().view(torch.uint8).numpy()


# ----------------------------------------------------------------------------- norm
def near(got, want, dtype, rel=2.0 ** -17, low=0.0):
    assert np.all(np.abs(f64(got) - want) <= np.abs(want) * (HALF[dtype] + rel) + LEAST[dtype] + low)


def run_norm(lib, x, w, r=None, eps=1e-6, offset=0.0, parts=("residual_out", "out", "out8"), shift=0):
    """add_rms_norm into fresh buffers (shift: elements that out starts behind an aligned address)."""
    rows, H = x.shape
    fresh = lambda dt: torch.empty(rows * H + shift, dtype=dt, device=DEV)[shift:].view(rows, H)  # noqa: E731
    o = {k: fresh(x.dtype) for k in ("residual_out", "out") if k in parts}
    if "out8" in parts:
        o["out8"] = torch.full((rows, H), 0x55, dtype=torch.uint8, device=DEV).view(F8)
        o["out8_scale"] = torch.empty(rows, rows8.blocks(H), device=DEV)
    lib.add_rms_norm(x, w, eps=eps, residual=r, weight_offset=offset, **o)
    torch.cuda.synchronize()
    return o


def check_norm(o, x, w, r=None, eps=1e-6, offset=0.0):
    h, y = rows8.add_rms_norm(f64(x), f64(w), eps, None if r is None else f64(r), offset)
    if "residual_out" in o:
        near(o["residual_out"], h, x.dtype, 2.0 ** -24)
    if "out" in o:
        near(o["out"], y, x.dtype, low=np.abs(f64(w) + offset) * 2.0 ** -150)
    if "out8" in o:
        H = x.shape[1]
        s = f64(o["out8_scale"])
        want = np.stack([np.abs(y[:, j * 128:(j + 1) * 128]).max(1) for j in range(rows8.blocks(H))], 1) / 448
        assert np.all(np.abs(s - want) <= want * 2.0 ** -16 + 2.0 ** -149)
        v = rows8.spread(bytes_of(o["out8"]), s, 1)
        per = np.repeat(s, 128, 1)[:, :H]
        assert np.all(np.abs(v - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * per) * (1 + 2.0 ** -13) + np.abs(y) * 2.0 ** -15
                      + (449 + np.abs(f64(w) + offset)) * 2.0 ** -150)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows, H", [(1, 5120), (3, 1), (2, 7), (5, 128), (1, 130), (64, 2573), (17, 8192), (2, 8200), (3, 16390), (2, 32768), (700, 1000)])
def test_norm(gpu_lib, rows, H, dtype):
    x, r, w = (rnd(*s, seed=H + k, dtype=dtype).to(DEV) for k, s in enumerate([(rows, H), (rows, H), (H,)]))
    check_norm(run_norm(gpu_lib, x, w, r), x, w, r)


def test_norm_parts(gpu_lib):
    """Every choice of outputs, with and without a residual, an offset, odd addresses, in place."""
    x, r, w = (rnd(*s, seed=k, dtype=torch.bfloat16).to(DEV) for k, s in enumerate([(9, 392), (9, 392), (392,)]))
    for parts in (("out",), ("out8",), ("residual_out",), ("residual_out", "out"), ("residual_out", "out8"), ("out", "out8")):
        for res in (r, None):
            check_norm(run_norm(gpu_lib, x, w, res, eps=1e-5, offset=1.0, parts=parts), x, w, res, 1e-5, 1.0)
    check_norm(run_norm(gpu_lib, x, w, r, shift=1), x, w, r)
    odd = torch.empty(9 * 392 + 3, dtype=torch.bfloat16, device=DEV)[3:].view(9, 392).copy_(x)
    check_norm(run_norm(gpu_lib, odd, w, r), x, w, r)
    for rows, H in ((9, 392), (3000, 640), (2500, 5120), (2000, 9000), (70, 17000), (1500, 333)):  # in place, more rows than are under way at once
        x, r, w = (rnd(*s, seed=k, dtype=torch.bfloat16).to(DEV) for k, s in enumerate([(rows, H), (rows, H), (H,)]))
        x2, r2 = x.clone(), r.clone()
        gpu_lib.add_rms_norm(x2, w, eps=1e-6, residual=r2, residual_out=r2, out=x2)
        check_norm(dict(residual_out=r2, out=x2), x, w, r)
        x2, r2 = x.clone(), r.clone()
        gpu_lib.add_rms_norm(x2, w, eps=1e-6, residual=r2, residual_out=x2, out=r2)
        check_norm(dict(residual_out=x2, out=r2), x, w, r)


@pytest.mark.parametrize("H", [100, 256, 512, 1032])
def test_huge_rows_among_others(gpu_lib, H):
    """Rows whose squares leave fp32's range beside rows whose do not, where several share a CTA."""
    x = rnd(2001, H, seed=H)
    x[::7] *= 1e30
    x[5, H // 2] = float("inf")
    x, w = x.to(DEV), rnd(H, seed=1).to(DEV)
    o = run_norm(gpu_lib, x, w, parts=("out", "out8"))
    fine = [i for i in range(2001) if i != 5]
    check_norm({k: v[fine] if v.dtype != F8 else v.view(torch.uint8)[fine].view(F8) for k, v in o.items()}, x[fine], w)
    assert torch.isnan(o["out"][5, H // 2]) and int(torch.isnan(o["out"][5]).sum()) == 1


def test_norm_values_at_the_ends(gpu_lib):
    """Rows of zeros, tiny, huge (squares beyond fp32), one loud feature; a NaN stays in its row, an infinity in its place."""
    x = rnd(9, 640, seed=5)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e25
    x[3, 7] = 3e38
    x[4] = 3e38
    x[5, 3] = float("nan")
    x[6, 600] = float("-inf")
    x[7] *= 2.0 ** -140
    x = x.to(DEV)
    w = rnd(640, seed=6).to(DEV)
    o = run_norm(gpu_lib, x, w, parts=("out", "out8"))
    fine = [0, 1, 2, 3, 4, 7, 8]
    check_norm({k: v[fine] if v.dtype != F8 else v.view(torch.uint8)[fine].view(F8) for k, v in o.items()}, x[fine], w)
    y, c, s = f64(o["out"]), bytes_of(o["out8"]), f64(o["out8_scale"])
    assert np.isnan(y[5]).all() and np.isnan(s[5]).all() and (c[5] & 0x7F == 0x7F).all()
    assert np.isnan(y[6, 600]) and (np.delete(y[6], 600) == 0).all() and np.isnan(s[6, 4]) and (s[6, :4] == 0).all() and (c[6, :512] & 0x7F == 0).all()


def test_quantize_is_exact(gpu_lib):
    """Codes and scales are whole decisions: equal to the oracle's, every type, odd lengths, odd addresses, wild values."""
    for k, (rows, H, dt) in enumerate([(1, 128, torch.bfloat16), (33, 5120, torch.bfloat16), (7, 2573, torch.float16), (5, 1, torch.float32),
                                       (4, 264, torch.float32), (129, 40, torch.float16), (2, 40000, torch.bfloat16)]):
        x = rnd(rows, H, seed=k).mul_(10.0 ** torch.linspace(-3, 3, rows)[:, None]).to(dt)
        x[0, : min(H, 128)] = 0
        for shift in (0, 1):
            d = torch.empty(rows * H + shift, dtype=dt, device=DEV)[shift:].view(rows, H).copy_(x)
            c, s = torch.empty(rows, H, dtype=torch.uint8, device=DEV), torch.empty(rows, rows8.blocks(H), device=DEV)
            gpu_lib.quantize_e4m3(d, c, s)
            torch.cuda.synchronize()
            wc, ws = rows8.quantize(x.float().numpy())
            assert np.array_equal(s.cpu().numpy(), ws)
            assert np.array_equal(rows8.decode(bytes_of(c)), rows8.decode(wc))
    x = torch.tensor([[1e-45] * 128 + [6e-43] * 128 + [float("nan")] + [1.0] * 127 + [float("inf")] + [1.0] * 127 + [3e38] * 128], device=DEV)
    c, s = torch.empty(1, 640, dtype=torch.uint8, device=DEV), torch.empty(1, 5, device=DEV)
    gpu_lib.quantize_e4m3(x, c, s)
    wc, ws = rows8.quantize(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(rows8.decode(bytes_of(c)), rows8.decode(wc), equal_nan=True)


# ----------------------------------------------------------------------------- products
def operands(rows, K, N, seed=0):
    g = np.random.default_rng(seed)
    byte = lambda *s: torch.from_numpy(rows8.encode(g.standard_normal(s) * g.choice([0.1, 30.0, 100.0], s)))  # noqa: E731
    a, w = byte(rows, K), byte(N, K)
    sa = torch.from_numpy(np.exp(g.uniform(-3, 3, (rows, rows8.blocks(K)))).astype(np.float32))
    sw = torch.from_numpy(np.exp(g.uniform(-6, 0, (rows8.blocks(N), rows8.blocks(K)))).astype(np.float32))
    return a, sa, w, sw


def product_bound(a, sa, w, sw):
    """What |out - exact| is at most, ahead of the output's rounding."""
    terms = np.abs(rows8.spread(a.numpy(), f64(sa), 1)) @ np.abs(rows8.spread(w.numpy(), f64(sw), 128)).T
    return terms * (128 * 2.0 ** -23 + (rows8.blocks(a.shape[1]) + 2) * 2.0 ** -24)


SIZES = [(1, 16, 1), (1, 128, 128), (1, 5120, 520), (2, 272, 129), (5, 1040, 1001), (16, 2048, 640), (17, 400, 130), (33, 384, 1000), (64, 6144, 256),
         (65, 640, 77), (128, 512, 384), (129, 4112, 260), (200, 256, 3000), (257, 144, 520), (400, 1024, 1024), (1, 2560, 20000), (1000, 128, 600),
         (3, 48, 40000), (96, 1280, 2000), (130, 20480, 130),
         # 64 columns shared by clusters of 8 and 4; CTA pairs, several rounds of them, ragged at both ends
         (1, 2112, 2666), (33, 2112, 2666), (20, 2384, 4997), (100, 3744, 2666), (1300, 272, 9000), (2500, 1040, 4999), (4100, 400, 5003)]


@pytest.mark.parametrize("rows, K, N", SIZES)
def test_matmul(gpu_lib, rows, K, N):
    a, sa, w, sw = operands(rows, K, N, seed=rows + K + N)
    want, bound = rows8.matmul(a.numpy(), sa.numpy(), w.numpy(), sw.numpy()), product_bound(a, sa, w, sw)
    d = [t.to(DEV) for t in (a, sa, w, sw)]
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        if dt == torch.float16 and np.abs(want).max() > 6e4:
            continue
        out = torch.full((rows + 1, N), float("nan"), dtype=dt, device=DEV)
        gpu_lib.matmul_e4m3(d[0].view(F8) if dt == torch.bfloat16 else d[0], d[1], d[2], d[3], out[:rows])
        torch.cuda.synchronize()
        got = f64(out)
        assert np.all(np.abs(got[:rows] - want) <= bound + np.abs(want) * HALF[dt] * (1 + 2.0 ** -10) + LEAST[dt]), (dt, np.abs(got[:rows] - want).max())
        assert np.isnan(got[rows]).all()  # nothing behind the last row
    again = torch.empty(rows, N, device=DEV)
    first = torch.empty(rows, N, device=DEV)
    gpu_lib.matmul_e4m3(*d, first)
    gpu_lib.matmul_e4m3(*d, again)
    assert torch.equal(first, again)
    arg, mx = torch.full((rows,), -7, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV)
    gpu_lib.matmul_e4m3_argmax(*d, arg, maxval=mx)
    assert torch.equal(mx, first.amax(1))
    i = arg.long().cpu().numpy()
    f = first.cpu().numpy()
    assert np.array_equal(i, np.argmax(f, 1))  # the lowest index of the largest


@pytest.mark.parametrize("rows, K, N", [(1, 256, 300), (16, 640, 4096), (48, 5120, 300), (300, 1152, 700)])
def test_matmul_of_whole_numbers_is_exact(gpu_lib, rows, K, N):
    g = np.random.default_rng(rows)
    ints = lambda *s: g.integers(-3, 4, s).astype(np.float64)  # noqa: E731
    a, w = ints(rows, K), ints(N, K)
    sa, sw = 2.0 ** g.integers(0, 3, (rows, rows8.blocks(K))), 2.0 ** g.integers(0, 3, (rows8.blocks(N), rows8.blocks(K)))
    ca, cw = rows8.encode(a), rows8.encode(w)
    out = torch.empty(rows, N, device=DEV)
    t = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    gpu_lib.matmul_e4m3(t(ca), t(sa.astype(np.float32)), t(cw), t(sw.astype(np.float32)), out)
    assert np.array_equal(f64(out), rows8.matmul(ca, sa, cw, sw))


def test_not_a_number_stays_in_its_row_and_column(gpu_lib):
    a, sa, w, sw = operands(40, 384, 260, seed=9)
    w[200, 5] = 0x7F
    sa[3, 1] = float("nan")
    a[7, 300] = 0xFF
    sw[1, 0] = float("inf")  # columns 128 .. 255
    d = [t.to(DEV) for t in (a, sa, w, sw)]
    out = torch.empty(40, 260, device=DEV)
    gpu_lib.matmul_e4m3(*d, out)
    bad = ~np.isfinite(f64(out))
    assert bad[3].all() and bad[7].all() and bad[:, 128:256].all()
    bad[[3, 7]] = False
    bad[:, 128:256] = False
    assert not bad.any()


def test_ties_take_the_lowest_index(gpu_lib):
    rows, K, N = 20, 256, 1500
    w = torch.full((N, K), 0x38, dtype=torch.uint8)  # every column the same
    a = torch.full((rows, K), 0x38, dtype=torch.uint8)
    a[5] = 0xB8
    sa, sw = torch.ones(rows, 2), torch.ones(rows8.blocks(N), 2)
    sw[5] = 2.0  # columns 640 .. 767 are larger, or smaller for row 5
    arg, mx = torch.empty(rows, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV)
    gpu_lib.matmul_e4m3_argmax(*[t.to(DEV) for t in (a, sa, w, sw)], arg, maxval=mx)
    want = np.full(rows, 640)
    want[5] = 0
    assert np.array_equal(arg.cpu().numpy(), want) and mx[5].item() == -256 and mx[0].item() == 512


@pytest.mark.parametrize("rows, H, V", [(1, 512, 5003), (3, 1040, 2000), (40, 272, 1000), (300, 640, 4100)])
def test_head(gpu_lib, rows, H, V):
    """bf16 rows through lm_head_logits and lm_head_argmax equal the calls one by one, bit for bit."""
    _, _, w, sw = (t.to(DEV) for t in operands(1, H, V, seed=V))
    h = rnd(rows, H, seed=1, dtype=torch.bfloat16).to(DEV)
    c, s = torch.empty(rows, H, dtype=F8, device=DEV), torch.empty(rows, rows8.blocks(H), device=DEV)
    gpu_lib.quantize_e4m3(h, c, s)
    one = torch.empty(rows, V, device=DEV)
    gpu_lib.matmul_e4m3(c, s, w, sw, one)
    logits = torch.empty(rows, V, device=DEV)
    gpu_lib.lm_head_logits(h, w.view(F8), logits, w_dtype=gpu_lib.E4M3_B128, V=V, scales=sw)
    assert torch.equal(logits, one)
    arg, mx = torch.empty(rows, dtype=torch.int32, device=DEV), torch.empty(rows, device=DEV)
    gpu_lib.lm_head_argmax(h, w, arg, w_dtype=gpu_lib.E4M3_B128, V=V, scales=sw, maxlogit=mx)
    assert np.array_equal(arg.cpu().numpy(), np.argmax(logits.cpu().numpy(), 1)) and torch.equal(mx, logits.amax(1))
    if rows * H < 16000:  # small enough for the calls without a workspace
        lib, again = gpu_lib.load(), torch.empty(rows, dtype=torch.int32, device=DEV)
        assert lib.tsv_lm_head_argmax_noalloc(h.data_ptr(), rows, H, V, gpu_lib.E4M3_B128, w.data_ptr(), sw.data_ptr(), None, again.data_ptr(),
                                              None, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(again, arg)


@pytest.mark.parametrize("rows, K, N", [(128, 5120, 100000), (100, 640, 40000), (300, 1152, 3000), (2048, 640, 20000), (33, 2112, 2666), (600, 7168, 512)])
def test_the_same_bits_every_time(gpu_lib, rows, K, N):
    """Many launches, back to back, while copies land in whatever order they do: a hand-off that relies on their order shows here."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    byte = lambda *s: torch.randint(0, 120, s, device=DEV, dtype=torch.uint8, generator=g)  # noqa: E731
    args = byte(rows, K), torch.rand(rows, rows8.blocks(K), device=DEV, generator=g), byte(N, K), torch.rand(rows8.blocks(N), rows8.blocks(K), device=DEV, generator=g)
    first, out = torch.empty(rows, N, device=DEV), torch.empty(rows, N, device=DEV)
    gpu_lib.matmul_e4m3(*args, first)
    for _ in range(12):
        out.zero_()
        for _ in range(8):
            gpu_lib.matmul_e4m3(*args, out)
        assert torch.equal(out, first)


def test_captured_and_on_two_streams(gpu_lib):
    """A norm, a product and an argmax recorded once and replayed on new inputs, and two streams at once."""
    rows, H, N = 24, 1024, 3000
    _, _, w, sw = (t.to(DEV) for t in operands(1, H, N, seed=2))
    wt = rnd(H, seed=3, dtype=torch.bfloat16).to(DEV)

    def buffers():
        return dict(x=torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV), c=torch.empty(rows, H, dtype=F8, device=DEV),
                    s=torch.empty(rows, 8, device=DEV), out=torch.empty(rows, N, dtype=torch.bfloat16, device=DEV),
                    arg=torch.empty(rows, dtype=torch.int32, device=DEV), ws=torch.empty(256, dtype=torch.uint8, device=DEV))

    def calls(b, stream=None):
        gpu_lib.add_rms_norm(b["x"], wt, eps=1e-6, out8=b["c"], out8_scale=b["s"], stream=stream)
        gpu_lib.matmul_e4m3(b["c"], b["s"], w, sw, b["out"], stream=stream)
        gpu_lib.matmul_e4m3_argmax(b["c"], b["s"], w, sw, b["arg"], workspace=b["ws"], stream=stream)

    b = buffers()
    calls(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(b)
    for seed in (1, 2):
        new = rnd(rows, H, seed=seed, dtype=torch.bfloat16).to(DEV)
        b["x"].copy_(new)
        g.replay()
        e = buffers()
        e["x"].copy_(new)
        calls(e)
        torch.cuda.synchronize()
        assert torch.equal(b["out"], e["out"]) and torch.equal(b["arg"], e["arg"])
    streams, sets = [torch.cuda.Stream(), torch.cuda.Stream()], [buffers(), buffers()]
    for q in sets:
        q["x"].copy_(new)
    torch.cuda.synchronize()
    for _ in range(10):
        for st, q in zip(streams, sets):
            calls(q, st)
    torch.cuda.synchronize()
    for q in sets:
        assert torch.equal(q["out"], e["out"]) and torch.equal(q["arg"], e["arg"])


def test_offsets_beyond_32_bits(gpu_lib):
    """Outputs, weights and rows that are longer than 2^31 elements, looked at near their ends."""
    rows, K, N = 17000, 16, 131072
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)  # 2.2e9 elements
    a = torch.full((rows, K), 0x38, dtype=torch.uint8, device=DEV)
    a[-1] = 0x40
    w = torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV)
    w[-1] = 0x48
    gpu_lib.matmul_e4m3(a, torch.ones(rows, 1, device=DEV), w, torch.ones(N // 128, 1, device=DEV), out)
    assert out[-1, -1].item() == 128 and out[-1, 0].item() == 32 and out[-2, -1].item() == 64 and (out[:, 5:-1:4097] [:-1] == 16).all()
    del out
    H = 32768
    x = torch.ones(70000, H, dtype=torch.bfloat16, device=DEV)  # 2.3e9 elements
    c, s = torch.empty(70000, H, dtype=torch.uint8, device=DEV), torch.empty(70000, 256, device=DEV)
    x[-1] = 3
    gpu_lib.quantize_e4m3(x, c, s)
    assert (c == 0x7E).all() and (s[-1].cpu() == float(np.float32(3) * rows8.INV_TOP)).all()
    gpu_lib.add_rms_norm(x, torch.ones(H, dtype=torch.bfloat16, device=DEV), eps=1e-6, out=x)
    assert (x[-3:] == 1).all() and (x[::777] == 1).all()
    one = torch.empty(1, 70000, device=DEV)
    gpu_lib.matmul_e4m3(c[:1], s[:1], c, torch.ones(547, 256, device=DEV), one)  # 2.3e9 weights
    assert (one == one[0, 0]).all()
