"""Pins of the recurrent layers' oracle and of the 4-bit cache format (CPU)."""
import numpy as np
import pytest

from oracle import append as oap
from oracle import gdn as og
from oracle import storage as osd


def inputs(rng, T, HK, HV, DK, DV):
    return (rng.standard_normal((T, HK, DK)), rng.standard_normal((T, HK, DK)), rng.standard_normal((T, HV, DV)),
            -rng.uniform(0.01, 1.0, (T, HV)), rng.uniform(0.1, 0.95, (T, HV)), rng.standard_normal((HV, DV, DK)))


def test_scan_is_the_product_of_its_transition_matrices():
    """S_n = S_0 A_1 ... A_n + sum_t b_t A_{t+1} ... A_n with A = e^g (I - beta k k^T) and b = beta v k^T."""
    rng = np.random.default_rng(0)
    q, k, v, g, beta, S0 = inputs(rng, 6, 1, 2, 8, 5)
    o, S = og.scan(q, k, v, g, beta, S0, norm_eps=0.0, scale=0.5)
    for h in range(2):
        want = S0[h]
        for t in range(6):
            A = np.exp(g[t, h]) * (np.eye(8) - beta[t, h] * np.outer(k[t, 0], k[t, 0]))
            want = want @ A + beta[t, h] * np.outer(v[t, h], k[t, 0])
            np.testing.assert_allclose(o[t, h], 0.5 * want @ q[t, 0], rtol=1e-10, atol=1e-10)
        np.testing.assert_allclose(S[h], want, rtol=1e-10, atol=1e-10)


def test_delta_rule_replaces_what_a_key_holds():
    """beta = 1, no decay, unit key: the state then returns exactly v for that key, whatever it held before."""
    rng = np.random.default_rng(1)
    k = rng.standard_normal((1, 1, 16))
    v = rng.standard_normal((1, 1, 4))
    S0 = rng.standard_normal((1, 4, 16))
    _, S = og.scan(k, k, v, np.zeros((1, 1)), np.ones((1, 1)), S0, norm_eps=1e-12)
    u = k[0, 0] / np.linalg.norm(k[0, 0])
    np.testing.assert_allclose(S[0] @ u, v[0, 0], atol=1e-9)
    w = rng.standard_normal(16)
    w -= (w @ u) * u  # other directions are untouched
    np.testing.assert_allclose(S[0] @ w, S0[0] @ w, atol=1e-9)


def test_gates():
    rng = np.random.default_rng(2)
    q, k, v, g, beta, S0 = inputs(rng, 1, 1, 1, 8, 8)
    _, S = og.scan(q, k, v, g, np.zeros((1, 1)), S0)  # beta 0 only forgets
    np.testing.assert_allclose(S, np.exp(g[0, 0]) * S0)
    a = og.scan(q, k, v, np.full((1, 1), -np.inf), beta, S0)
    b = og.scan(q, k, v, g, beta, np.zeros_like(S0))  # forgetting everything is starting from nothing
    np.testing.assert_allclose(a[0], b[0])
    np.testing.assert_allclose(a[1], b[1])


@pytest.mark.parametrize("seed", range(4))
def test_every_tree_node_is_its_own_root_path(seed):
    rng = np.random.default_rng(seed)
    T = 9
    par = [-1] + [int(rng.integers(0, i)) for i in range(1, T)]
    q, k, v, g, beta, S0 = inputs(rng, T, 2, 4, 8, 6)
    o = og.tree_verify(q, k, v, g, beta, S0, par)
    for i in range(T):
        path = [i]
        while par[path[0]] >= 0:
            path.insert(0, par[path[0]])
        want, S = og.scan(q[path], k[path], v[path], g[path], beta[path], S0)
        np.testing.assert_allclose(o[i], want[-1], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(og.commit(q, k, v, g, beta, S0, path), S, rtol=1e-12, atol=1e-12)


def test_value_heads_read_their_group_of_key_heads():
    rng = np.random.default_rng(5)
    q, k, v, g, beta, S0 = inputs(rng, 4, 2, 6, 8, 8)
    o, S = og.scan(q, k, v, g, beta, S0)
    rq, rk = np.repeat(q, 3, axis=1), np.repeat(k, 3, axis=1)
    o2, S2 = og.scan(rq, rk, v, g, beta, S0)
    np.testing.assert_allclose(o, o2)
    np.testing.assert_allclose(S, S2)


def test_four_bit_cache_row_by_hand():
    # low nibble first; scale 0.5, bias -1: codes 1, 2, ..., on a group of 64
    packed = np.zeros((1, 32), dtype=np.uint8)
    packed[0, 0] = 0x21
    packed[0, 31] = 0xF0
    pair = np.array([[[0x3800, 0xBC00]]], dtype=np.uint16)
    x = osd.kv_values(4, packed, pair)
    assert x[0, :4].tolist() == [-0.5, 0.0, -1.0, -1.0] and x[0, 62:].tolist() == [-1.0, 6.5]
    two = osd.int4_affine(np.zeros((1, 64), dtype=np.uint8), np.array([[[0, 0x3C00], [0, 0x4000]]], dtype=np.uint16))
    assert two[0, 63] == 1.0 and two[0, 64] == 2.0


def test_four_bit_quantisation_by_hand():
    x = np.zeros(64)
    x[0], x[1], x[2], x[3] = -1.0, 14.0, 0.5, 1.5  # range 15: scale 1, bias -1
    codes, pair = oap.quantize_token4(x)
    assert pair.tolist() == [[0x3C00, 0xBC00]]
    assert codes[:5].tolist() == [0, 15, 2, 2, 1]  # 1.5 and 2.5 round to even
    codes, pair = oap.quantize_token4(np.full(64, 3.0))  # a single value: scale 0, the bias holds it
    assert codes.tolist() == [0] * 64 and pair.tolist() == [[0, 0x4200]]
    codes, pair = oap.quantize_token4(np.concatenate([np.full(32, -1e30), np.full(32, 1e30)]))
    # cut to +-65000: 8666.67 to the nearest 8, -65000 to the nearest 32 (to even); every value is finite in fp16
    assert osd.f16(pair).tolist() == [[8664.0, -64992.0]] and codes[0] == 0 and codes[63] == 15
    assert -64992.0 + 15 * 8664.0 < 65504.0
    x = np.full(64, np.nan)
    x[5], x[9] = np.inf, 1.0
    codes, pair = oap.quantize_token4(x)
    assert osd.f16(pair).tolist()[0][1] == 1.0 and codes[5] == 15 and codes[9] == 0 and codes[0] == 0
    codes, pair = oap.quantize_token4(np.full(64, np.nan))
    assert np.isfinite(osd.f16(pair)).all() and codes.tolist() == [0] * 64


@pytest.mark.parametrize("seed", range(3))
def test_four_bit_quantisation_error(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal(256) * 3).astype(np.float32).astype(np.float64)
    codes, pair = oap.quantize_token4(x)
    p = codes[0::2] | (codes[1::2] << 4)
    y = osd.kv_values(4, p.astype(np.uint8), pair)
    s = np.repeat(osd.f16(pair[:, 0]), 64)
    # half a step, plus the fp16 rounding of the range (15 steps) and of the minimum (half of 2^-10 each)
    assert np.all(np.abs(x - y) <= s / 2 + 15 * s * 2.0 ** -10 + np.abs(x).max() * 2.0 ** -11)
