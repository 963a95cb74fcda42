"""CPU pins of the serving operators' oracle."""
import numpy as np
import pytest

from oracle import serving_ref as o


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_is_the_complex_product(layout):
    g = np.random.default_rng(1)
    x, pos, table = g.normal(size=(5, 2, 16)), [0, 3, 9, 1, 7], o.rope_table(10, 12)
    y = o.rope(x, pos, table, layout)
    for t, p in enumerate(pos):
        for i, w in enumerate(o.rope_frequencies(12)):
            ia, ib = (i, i + 6) if layout == "half" else (2 * i, 2 * i + 1)
            z = (x[t, :, ia] + 1j * x[t, :, ib]) * np.exp(1j * p * w)
            assert np.allclose(y[t, :, ia], z.real, atol=1e-13) and np.allclose(y[t, :, ib], z.imag, atol=1e-13)
    assert np.array_equal(y[..., 12:], x[..., 12:])
    assert np.allclose(o.rope(y, pos, table, layout, inverse=True), x, atol=1e-13)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_rope_is_the_gradient(layout):
    g = np.random.default_rng(2)
    x, w = g.normal(size=(3, 2, 8)), g.normal(size=(3, 2, 8))
    pos, table = [4, 0, 6], o.rope_table(8, 6)
    grad = o.rope(w, pos, table, layout, inverse=True)
    for _ in range(10):
        d = g.normal(size=x.shape)
        diff = ((o.rope(x + 1e-4 * d, pos, table, layout) - o.rope(x - 1e-4 * d, pos, table, layout)) * w).sum() / 2e-4
        assert abs(diff - (grad * d).sum()) < 1e-8


def test_rope_scalings():
    w = o.rope_frequencies(64)
    assert np.allclose(o.rope_frequencies(64, scaling=dict(kind="linear", factor=4.0)), w / 4)
    b = o.rope_frequencies(64, scaling=dict(kind="base", factor=4.0))
    assert b[0] == 1.0 and np.isclose(b[-1], w[-1] / 4)  # the slowest pair reaches as if all were divided
    p = o.rope_frequencies(64, scaling=dict(kind="parts", factor=4.0, original=2048))
    turns = 2048 * w / (2 * np.pi)
    assert np.allclose(p[turns >= 32], w[turns >= 32]) and np.allclose(p[turns <= 1], w[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(p[mid] < w[mid]) and np.all(p[mid] > w[mid] / 4)


@pytest.mark.parametrize("bits", [4, 8])
def test_grid_error_is_half_a_step(bits):
    g = np.random.default_rng(bits)
    for row in (g.normal(size=64), np.abs(g.normal(size=64)), -np.abs(g.normal(size=64)), 1e-25 * g.normal(size=64)):
        s, z, q = o.kv_grid(row, bits)
        assert q.max() <= (1 << bits) - 1
        assert np.abs(o.kv_values(s, z, q) - row).max() <= float(s) * (1.0 + 1e-5)  # half from the code, half from z
    assert o.kv_grid(np.zeros(64), bits)[0] == 1 and not o.kv_grid(np.zeros(64), bits)[2].any()
    assert np.isnan(o.kv_grid(np.array([1.0, np.inf]), bits)[0]) and np.isnan(o.kv_grid(np.array([np.nan]), bits)[0])
    assert np.isnan(o.kv_grid(np.array([3e38, -3e38]), bits)[0])
    s, z, q = o.kv_grid(np.array([1e-32, -1e-32]), bits)
    assert s == 1 and not o.kv_values(s, z, q).any()


@pytest.mark.parametrize("bits", [4, 8])
def test_pool_round_trip_and_attention(bits):
    g = np.random.default_rng(bits)
    pool = o.empty_pool(3, 2, 16, 64, bits)
    k, v = g.normal(size=(20, 2, 64)), g.normal(size=(20, 2, 64))
    slots = g.permutation(48)[:20]
    slots[3] = -1
    o.kv_write(pool, k, v, slots, bits)
    kr, vr = o.kv_read(pool, slots, bits)
    assert not kr[3].any() and not vr[3].any()
    for t in range(20):
        for h in range(2):
            if t != 3:
                assert np.array_equal(kr[t, h], o.kv_values(*o.kv_grid(k[t, h], bits)))
                assert np.array_equal(vr[t, h], o.kv_values(*o.kv_grid(v[t, h], bits)))
    # positions 0..19 of one sequence in pages 2, 0: attention equals the dense softmax
    slots = np.concatenate([32 + np.arange(16), np.arange(4)])
    o.kv_write(pool, k, v, slots, bits)
    kr, vr = (x.astype(np.float64) for x in o.kv_read(pool, slots, bits))
    q = g.normal(size=(1, 3, 4, 64))
    mask = np.array([[[0b001], [0b011], [0b000]]])
    got, spread, top = o.tree_attention(q, pool, np.array([[2, 0]]), [17], bits, mask)
    for t, seen in enumerate([list(range(18)), list(range(19)), list(range(17))]):
        for h in range(4):
            e = np.exp(kr[seen, h // 2] @ q[0, t, h] / 8)
            # the dense values are rounded to float32, the oracle's are not
            assert np.allclose(got[0, t, h], (e[:, None] * vr[seen, h // 2]).sum(0) / e.sum(), rtol=0, atol=1e-6)
    assert np.all(spread >= np.abs(got)) and top.shape == (1, 3, 4, 2)
    chain, _, _ = o.tree_attention(q, pool, np.array([[2, 0]]), [17], bits)
    full, _, _ = o.tree_attention(q, pool, np.array([[2, 0]]), [17], bits, np.array([[[1], [3], [7]]]))
    assert np.array_equal(chain, full)
    assert not o.tree_attention(q, pool, np.array([[2, 0]]), [-1], bits)[0].any()
    assert not o.tree_attention(q, pool, np.array([[-1, 7]]), [17], bits)[0].any()
