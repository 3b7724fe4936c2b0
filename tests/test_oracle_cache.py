"""The cache oracle against hand-worked grids, exact arithmetic and a direct softmax."""
from fractions import Fraction

import numpy as np
import pytest

import oracle


def test_bf16_up_is_the_next_value_up():
    assert oracle.bf16_up(np.float32(1.0)) == 1.0
    assert oracle.bf16_up(np.float32(1.0) + np.float32(2 ** -23)) == 1.0 + 2 ** -7
    x = np.abs(np.random.default_rng(0).standard_normal(1000)).astype(np.float32)
    up = oracle.bf16_up(x)
    assert np.all(up >= x) and np.all(up <= x * (1 + 2.0 ** -7))
    assert np.all(up.view(np.uint32) & 0xFFFF == 0)


def test_grid_by_hand():
    """[-1, 0, 0.5, 2] at 4 bits: step 3/15 = 0.2, up to bf16 205/1024; z = rint(4.995) = 5."""
    x = np.zeros(32, np.float32)
    x[:4] = [-1.0, 0.0, 0.5, 2.0]
    q, s, z = oracle.grid_quantize(x, 4, 32)
    assert s[0] == np.float32(205 / 1024) and z[0] == 5
    assert list(q[:4]) == [0, 5, 7, 15]
    assert np.all(q[4:] == 5)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_grid_covers_its_group(bits, group):
    """Every value is within half a step of what its code stands for (plus fp32 rounding), and the
    zero is on the grid."""
    rng = np.random.default_rng(group + bits)
    x = (rng.standard_normal((50, 128)) * np.exp2(rng.uniform(-20, 20, (50, 1)))) \
        .astype(np.float32)
    q, s, z = oracle.grid_quantize(x, bits, group)
    v = oracle.cache_values(q, s, z)
    step = np.repeat(s.astype(np.float64), group, -1)
    # at the ends z's own rounding can cost another half step, never more
    assert np.all(np.abs(v - x) <= step * (1.0 + 2.0 ** -20))
    q0, _, _ = oracle.grid_quantize(np.zeros((1, 128), np.float32), bits, group)
    assert len(set(q0.ravel())) == 1


def test_values_are_exact():
    q = np.array([[0, 3, 15, 7] * 8], np.uint8)
    s, z = np.array([[0.201171875]], np.float32), np.array([[5]], np.uint8)
    v = oracle.cache_values(q, s, z)
    for a, c in zip(v.ravel(), q.ravel()):
        assert Fraction(a) == Fraction(0.201171875) * (int(c) - 5)


def test_not_finite_groups_read_as_nan():
    x = np.ones((4, 64), np.float32)
    x[0, 3], x[1, 40], x[2, 0], x[3, :2] = np.nan, np.inf, -np.inf, [3e38, -3e38]
    q, s, z = oracle.grid_quantize(x, 4, 32)
    bad = np.isnan(s)
    assert bad.tolist() == [[True, False], [False, True], [True, False], [True, False]]
    assert np.all(q.reshape(4, 2, 32)[bad] == 0) and np.all(z[bad] == 0)


def test_pack_rows_nibbles():
    codes = np.arange(16, dtype=np.uint8)[None]
    assert oracle.pack_rows(codes, 4).tolist() == [[0x76543210, 0xFEDCBA98]]
    assert oracle.pack_rows(codes[:, :4] * 16, 8).tolist() == [[0x30201000]]


def test_attend_against_a_direct_softmax():
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((7, 64)), rng.standard_normal((7, 64)), rng.standard_normal(64)
    w = np.exp(0.125 * (k @ q))
    assert np.allclose(oracle.attend(q, k, v, 0.125), (w[:, None] * v).sum(0) / w.sum(), rtol=1e-12)
    assert np.all(oracle.attend(q, k[:0], v[:0], 0.125) == 0)
    c = [oracle.grid_quantize(t.astype(np.float32), 8, 64) for t in (k, v)]
    out, tol = oracle.attend_bound(q, *c[0], *c[1], 0.125)
    ref = oracle.attend(q, oracle.cache_values(*c[0]), oracle.cache_values(*c[1]), 0.125)
    assert np.allclose(out, ref, rtol=1e-12) and np.all(tol > 0) and np.all(tol < 0.02)


def test_bound_catches_a_misplaced_token():
    """A kernel that met one token more, one fewer, or another's value leaves the bound: planted in
    the oracle's inputs."""
    rng = np.random.default_rng(4)
    q = rng.standard_normal(128)
    k = oracle.grid_quantize(rng.standard_normal((90, 128)).astype(np.float32), 4, 128)
    v = oracle.grid_quantize(rng.standard_normal((90, 128)).astype(np.float32), 4, 128)
    out, tol = oracle.attend_bound(q, *k, *v, 128 ** -0.5)
    for wrong in (slice(0, 89), list(range(90)) + [3], [1] + list(range(1, 90))):
        o2, _ = oracle.attend_bound(q, *(a[wrong] for a in k), *(a[wrong] for a in v), 128 ** -0.5)
        assert np.any(np.abs(o2 - out) > 2 * tol)
