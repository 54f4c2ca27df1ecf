"""Pins of the cache oracle on the CPU, each against something that shares no
code with it."""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache_oracle as co


def test_e4m3_values_and_rounding_equal_torch():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, co.E4M3, equal_nan=True)
    g = np.random.default_rng(1)
    x = np.concatenate([g.normal(size=4000) * 2.0 ** g.integers(-14, 9, 4000),
                        co.E4M3[:127], (co.E4M3[1:127] + co.E4M3[:126]) / 2])  # ties
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(co.e4m3_round(x), want)
    assert co.e4m3_round(np.array([1e9, -np.inf])).tolist() == [448.0, -448.0]


def test_block_scale_is_the_smallest_power_of_two_that_fits():
    for top, want in [(448.0, 1.0), (448.1, 2.0), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7),
                      (0.0, 2.0 ** -126), (1e-44, 2.0 ** -126)]:
        assert co.block_scale(np.array([0.0, -top])) == want
    assert co.block_scale(np.array([np.inf, 3.0, np.nan])) == co.block_scale(np.array([3.0]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("per_axis", [False, True])
def test_rotary_is_a_complex_product(interleaved, per_axis):
    g = np.random.default_rng(2)
    X = g.normal(size=(2, 3, 5, 14))
    sections, P = [2, 1, 3], 6
    pos = g.integers(-50, 50, (3, 2, 5))
    f = np.array(co.rotary_frequencies(sections, 100.0, per_axis))
    Y = co.rotary(X, pos, f, sections, interleaved)
    ia, ib = (np.arange(P) * 2, np.arange(P) * 2 + 1) if interleaved else \
        (np.arange(P), np.arange(P) + P)
    axis = np.repeat(np.arange(3), sections)
    turn = np.exp(1j * np.moveaxis(pos[axis], 0, -1) * f)[:, None]
    z = (X[..., ia] + 1j * X[..., ib]) * turn
    assert np.allclose(Y[..., ia], z.real, atol=1e-12)
    assert np.allclose(Y[..., ib], z.imag, atol=1e-12)
    assert np.array_equal(Y[..., 12:], X[..., 12:])
    back = co.rotary(Y, pos, f, sections, interleaved, inverse=True)
    assert np.allclose(back, X, atol=1e-12)


def test_rotary_scores_depend_on_the_distance_alone():
    g = np.random.default_rng(3)
    q, k = g.normal(size=(1, 1, 1, 8)), g.normal(size=(1, 1, 1, 8))
    f = co.rotary_frequencies([4])
    at = lambda x, p: co.rotary(x, np.full((1, 1, 1), p), f, [4])
    a = (at(q, 17) * at(k, 5)).sum()
    b = (at(q, 112) * at(k, 100)).sum()
    assert abs(a - b) < 1e-12


def test_reserve_serves_in_order_and_skips_what_does_not_fit():
    table = np.full((4, 4), -1)
    table[1, 0] = 9
    total, slots, left, after, full, bad = co.reserve(
        [0, 3, 0, 2], [5, 1, 12, 1], [30, 31, 32], 3, [list(r) for r in table], 4, 12)
    # item 0 takes 2 blocks from the top, item 1 fits its old block, item 2
    # needs 3 more, item 3 needs none
    assert total == [5, 4, 0, 3] and left == 1 and full and not bad
    assert after[0, :2].tolist() == [32, 31] and after[1, 0] == 9
    assert slots[0, :6].tolist() == [128, 129, 130, 131, 124, -1] and slots[1, 0] == 39
    assert (slots[2] == -1).all()


def test_append_then_attention_is_dense_attention_of_the_rounded_rows():
    """Rows written block by block through a shuffled table, read back and
    attended to, against the dense decode oracle on rows rounded directly."""
    g = np.random.default_rng(4)
    B, h, n, d, bt = 2, 2, 37, 16, 16
    K, V = g.normal(size=(B, h, n, d)), g.normal(size=(B, h, n, d)) * 3
    table = np.array([[4, 0, 2], [1, 5, 3]])
    codes = [np.zeros((6, h, bt, d)) for _ in range(2)]
    scale = [np.ones((6, h)) for _ in range(2)]
    pos = np.arange(n)
    slots = table[:, pos // bt] * bt + pos % bt
    for x, c, s in zip((K, V), codes, scale):
        co.append(x, slots, c, s, bt)
    def rounded(x):
        y = np.empty_like(x)
        for j in range(0, n, bt):
            s = np.abs(x[:, :, j:j + bt]).max(axis=(2, 3)) / 448
            s = 2.0 ** np.ceil(np.log2(s))[:, :, None, None]
            y[:, :, j:j + bt] = s * torch.from_numpy(x[:, :, j:j + bt] / s).to(
                torch.float8_e4m3fn).double().numpy()
        return y
    Q = g.normal(size=(B, h, 3, d))
    for tail in (False, True):
        Z, (A, _, _, _) = co.attention_cache(Q, codes[0], codes[1], scale[0], scale[1], table, [n, n],
                                     [3, 3], 0.25, tail)
        ref = oracle.attention_decode(Q, rounded(K), rounded(V), 0.25, [n, n], tail)
        assert np.allclose(Z, ref, atol=1e-12)
        assert (A >= np.abs(Z) - 1e-12).all()


def test_appending_in_two_calls_rounds_kept_rows_to_the_larger_scale():
    codes, scale = np.zeros((1, 1, 16, 2)), np.zeros((1, 1))
    slots = np.arange(2)[None]
    co.append(np.array([[[[1.0, 0.001]]]]), slots[:, :1], codes, scale, 16)
    assert scale[0, 0] == 2.0 ** -8
    small = codes[0, 0, 0, 1] * scale[0, 0]
    assert abs(small - 0.001) <= 0.001 * 2 ** -4
    co.append(np.array([[[[100.0, 5.0]]]]), slots[:, 1:], codes, scale, 16)
    assert scale[0, 0] == 2.0 ** -2 and codes[0, 0, 0, 0] == 4.0
    # 0.001 is 2.05 times 2^-9 s: below the normal numbers only multiples are left
    assert codes[0, 0, 0, 1] * scale[0, 0] == 2 * 2.0 ** -11
