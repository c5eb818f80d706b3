"""Pins of the 8-bit rows' oracle: values worked by hand, torch's own conversions, properties."""
import numpy as np
import pytest
import torch

from oracle import rows8


def test_codes_by_hand():
    t = rows8.TABLE
    assert [t[0x00], t[0x01], t[0x07], t[0x08], t[0x38], t[0x39], t[0x7E], t[0xB8]] == \
        [0.0, 2.0 ** -9, 7 * 2.0 ** -9, 2.0 ** -6, 1.0, 1.125, 448.0, -1.0]
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF]) and np.isfinite(np.delete(t, [0x7F, 0xFF])).all()
    # halfway between two codes goes to the even mantissa: 1.0625 is between 1.0 (0x38) and 1.125 (0x39)
    assert rows8.encode([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 1e9, -1e9, np.nan, -0.0]).tolist() == \
        [0x38, 0x3A, 0x00, 0x02, 0x7E, 0xFE, 0x7F, 0x80]


def test_conversions_are_torchs():
    every = torch.arange(256, dtype=torch.uint8)
    v = every.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(v, rows8.TABLE, equal_nan=True)
    x = torch.from_numpy(np.random.default_rng(1).uniform(-448, 448, 20000).astype(np.float32))
    x[:5000] *= 2.0 ** -14
    assert np.array_equal(x.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), rows8.encode(x.numpy()))


def test_groups():
    x = np.zeros((2, 300), np.float32)
    x[0, 5], x[0, 130], x[1, 299] = 448.0, -1.0, 3.5
    codes, scale = rows8.quantize(x)
    assert scale.shape == (2, 3) and scale[0].tolist() == [1.0, np.float32(1) / np.float32(448), 0.0]
    assert codes[0, 5] == 0x7E and codes[0, 130] == 0xFE and codes[1, 299] == 0x7E and (codes != 0).sum() == 3
    y = np.random.default_rng(0).standard_normal((4, 300)).astype(np.float32)
    codes, scale = rows8.quantize(y)
    step = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * np.repeat(scale, 128, 1)[:, :300]) * (1 + 2.0 ** -20)
    assert (np.abs(rows8.spread(codes, scale, 1) - y) <= step).all()


def test_norm_is_torchs():
    rng = np.random.default_rng(2)
    x, r, w = rng.standard_normal((5, 37)), rng.standard_normal((5, 37)), rng.standard_normal(37)
    h, y = rows8.add_rms_norm(x, w, 1e-5, r, 1.0)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (37,), torch.from_numpy(1 + w), 1e-5)
    assert np.array_equal(h, x + r) and np.allclose(y, ref.numpy(), rtol=1e-13)
    assert np.allclose(rows8.add_rms_norm([[3.0, 4.0]], [1.0, 2.0], 0.0)[1], [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])


def test_product_by_blocks():
    rng = np.random.default_rng(3)
    a, w = rng.integers(0, 0x7F, (3, 272)).astype(np.uint8), rng.integers(0, 0x7F, (130, 272)).astype(np.uint8)
    sa, sw = rng.uniform(1, 2, (3, 3)), rng.uniform(1, 2, (2, 3))
    out = rows8.matmul(a, sa, w, sw)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        want = sum(sa[m, b] * sw[n // 128, b] * (rows8.TABLE[a[m, b * 128:(b + 1) * 128]] * rows8.TABLE[w[n, b * 128:(b + 1) * 128]]).sum()
                   for b in range(3))
        assert out[m, n] == pytest.approx(want, rel=1e-12)


def test_logprobs():
    got = rows8.logprobs([[0.0, np.log(3.0), 0.0, -np.inf]], targets=[2], top_k=4)
    assert np.allclose(got["logp"], np.log(0.2)) and got["rank"][0] == 2 and got["top_tokens"][0].tolist() == [1, 0, 2, 3]
    assert np.allclose(got["entropy"], -(0.6 * np.log(0.6) + 0.4 * np.log(0.2))) and got["top_logp"][0, 3] == -np.inf
    x = np.random.default_rng(4).standard_normal((3, 50))
    got = rows8.logprobs(x, [0, 49, -1], 0.5, 3)
    ref = torch.log_softmax(torch.from_numpy(x) / 0.5, 1).numpy()
    assert np.allclose(got["logp"][:2], [ref[0, 0], ref[1, 49]]) and np.isnan(got["logp"][2]) and got["rank"][2] == -1
    assert np.allclose(got["top_logp"], -np.sort(-ref, 1)[:, :3])
    for bad in ([np.nan, 1.0], [np.inf, 1.0], [-np.inf, -np.inf]):
        got = rows8.logprobs([bad], [1], 1.0, 1)
        assert np.isnan(got["logp"][0]) and np.isnan(got["entropy"][0]) and got["top_tokens"][0, 0] == -1 and got["rank"][0] == -1
