"""Pins of the 4-bit KV cache's oracle: hand-worked rows, closed forms of the
attention, finite differences of its log-sum, brute force for the eviction."""
import itertools

import numpy as np
import pytest

import oracle


def test_encode_hand_worked_block():
    # amax 12, S 1: scale E4M3(2) = 0x40; 12 / 2 = 6, -3 / 2 = -1.5, 1.5 / 2 = 0.75 -> 1 (even)
    x = np.zeros((1, 16), np.float32)
    x[0, :4] = [12, -3, 1.5, -0.25]
    codes, scales = oracle.kv4_encode(x, 1.0)
    assert scales[0, 0] == 0x40
    assert list(codes[0, :2]) == [0x7 | (0xB << 4), 0x2 | (0x8 << 4)]
    assert list(oracle.kv4_decode(codes, scales, 1.0)[0, :4]) == [12, -3, 2, 0]


def test_encode_agrees_with_the_residual_quantiser():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 64)).astype(np.float32)
    codes, scales, S = oracle.nvfp4_quantize(x)
    c2, s2 = oracle.kv4_encode(x, S)
    assert np.array_equal(codes, c2) and np.array_equal(scales, s2)


def test_encode_zero_inf_and_nan():
    x = np.zeros((3, 16), np.float32)
    x[1, 0], x[1, 1] = np.inf, -np.inf
    x[2, 0], x[2, 1] = np.nan, 6.0
    codes, scales = oracle.kv4_encode(x, 1.0)
    v = oracle.kv4_decode(codes, scales, 1.0)
    assert np.all(v[0] == 0) and list(v[1, :2]) == [2688.0, -2688.0]
    assert list(v[2, :2]) == [6.0, 6.0]


@pytest.mark.parametrize("S", [1.0, 0.25, 0.1])
def test_encode_error_is_within_a_step(S):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 128)).astype(np.float32)
    v = oracle.kv4_decode(*oracle.kv4_encode(x, S), S)
    amax = np.abs(x.reshape(64, 8, 16)).max(-1).repeat(16, -1)
    # a step of E2M1 is at most 2 of 6, and the scale is within 2^-4 of amax / 6
    assert np.all(np.abs(v - x) <= amax * (1 / 6 + 1 / 16) + 1e-6)


def _toy(seed=3, B=2, T=3, Hq=4, Hkv=2, N=7, dh=16):
    rng = np.random.default_rng(seed)
    Q, K = rng.standard_normal((B, T, Hq, dh)), rng.standard_normal((B, Hkv, N, dh))
    return Q, K, rng.standard_normal((B, Hkv, N, dh))


def test_equal_scores_give_the_mean_and_log_n():
    Q, K, V = _toy()
    s = oracle.kv4_scores(0 * Q, K, 1.0, length=[5, 7])
    O, lse = oracle.kv4_attention(s, V)
    assert np.allclose(lse[0], np.log(5)) and np.allclose(lse[1], np.log(7))
    assert np.allclose(O[0, 0, 3], V[0, 1, :5].mean(0)) and np.allclose(O[1, 2, 0], V[1, 0].mean(0))


def test_one_visible_slot_gives_its_row():
    Q, K, V = _toy()
    span = np.tile([4, 5], (2, 3, 1))
    s = oracle.kv4_scores(Q, K, 0.5, span=span)
    O, lse = oracle.kv4_attention(s, V)
    assert np.allclose(O[1, 2, 3], V[1, 1, 4])
    assert np.allclose(lse[0, 1, 0], 0.5 * Q[0, 1, 0] @ K[0, 0, 4])


def test_rows_that_see_nothing():
    Q, K, V = _toy()
    s = oracle.kv4_scores(Q, K, 1.0, length=[0, 7], span=np.tile([3, 3], (2, 3, 1)))
    O, lse = oracle.kv4_attention(s, V)
    assert np.all(O == 0) and np.all(np.isneginf(lse))
    assert np.all(oracle.kv4_weight(s, lse, 2) == 0)


def test_value_gradient_of_the_log_sum_is_the_output():
    """d lse / d s_n = p_n: by central differences, which ties O, lse and the
    weight to each other."""
    Q, K, V = _toy(B=1, T=1, Hq=1, Hkv=1)
    s = oracle.kv4_scores(Q, K, 0.7)
    O, lse = oracle.kv4_attention(s, V)
    p = oracle.kv4_weight(s, lse, 1)[0, 0]
    for n in range(7):
        up, dn = s.copy(), s.copy()
        up[..., n] += 1e-5
        dn[..., n] -= 1e-5
        g = (oracle.kv4_attention(up, V)[1] - oracle.kv4_attention(dn, V)[1]) / 2e-5
        assert abs(g[0, 0, 0] - p[n]) < 1e-9
    assert np.allclose(p @ V[0, 0], O[0, 0, 0]) and abs(p.sum() - 1) < 1e-12


def test_cap_bias_and_positions():
    Q, K, _ = _toy(N=4)
    kpos = np.tile([9, 2, 5, 0], (2, 2, 1))
    qpos = np.tile([1, 4, 8], (2, 1))
    slope = np.array([0.5, 0.0, 1.0, 2.0])
    raw = oracle.kv4_scores(Q, K, 3.0)
    s = oracle.kv4_scores(Q, K, 3.0, kpos=kpos, qpos=qpos, slope=slope, cap=2.0,
                          span=np.tile([2, 9], (2, 3, 1)))
    assert np.all(np.isneginf(s[..., 0])) and np.all(np.isneginf(s[..., 3]))
    assert np.isclose(s[0, 1, 2, 2], 2 * np.tanh(raw[0, 1, 2, 2] / 2) - abs(4 - 5))
    assert np.isclose(s[1, 2, 3, 1], 2 * np.tanh(raw[1, 2, 3, 1] / 2) - 2 * abs(8 - 2))


def test_weight_sums_to_the_number_of_rows():
    Q, K, V = _toy()
    s = oracle.kv4_scores(Q, K, 1.0, length=[3, 7])
    w = oracle.kv4_weight(s, oracle.kv4_attention(s, V)[1], 2)
    assert np.allclose(w.sum(-1), 3 * 2) and np.all(w[0, :, 3:] == 0)


def test_keep_matches_brute_force():
    """Among all sets with the protected slots, the kept one has the largest
    weight and, of those, the lowest slots."""
    rng = np.random.default_rng(5)
    for _ in range(40):
        n, sink, recent = 9, int(rng.integers(0, 3)), int(rng.integers(0, 3))
        keep = int(rng.integers(max(1, sink + recent), 9))
        w = rng.integers(0, 4, n).astype(np.float32)      # many ties
        need = set(range(sink)) | set(range(n - recent, n))
        best = max((sum(w[list(c)]), [-i for i in c])
                   for c in itertools.combinations(range(n), keep) if need <= set(c))
        assert [-i for i in best[1]] == list(oracle.kv4_keep(w, n, keep, sink, recent))


def test_keep_short_and_nan():
    w = np.array([np.nan, 1, -np.inf, 2, np.nan], np.float32)
    assert list(oracle.kv4_keep(w, 3, 4, 0, 0)) == [0, 1, 2]
    assert list(oracle.kv4_keep(w, 5, 3, 0, 0)) == [1, 2, 3]
    assert list(oracle.kv4_keep(w, 5, 4, 0, 0)) == [0, 1, 2, 3]
