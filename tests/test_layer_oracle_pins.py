"""The 4-bit layer's oracle, pinned by hand-computed values and by invariants (CPU)."""
import numpy as np
import pytest

import oracle.layer_oracle as O


def test_e2m1_rounding_by_hand():
    # value: nearest level; a tie goes to the even code (levels 0, 1, 2, 4 have even codes)
    pins = {0.0: 0, 0.24: 0, 0.25: 0, 0.26: 0.5, 0.74: 0.5, 0.75: 1, 1.25: 1, 1.26: 1.5, 1.75: 2, 2.5: 2, 2.51: 3,
            3.5: 4, 3.49: 3, 5.0: 4, 5.01: 6, 6.0: 6, 7.9: 6, 1e30: 6}
    got = O.E2M1[O.nearest_code(np.array(list(pins)), O.E2M1)]
    np.testing.assert_array_equal(got, np.array(list(pins.values()), float))


def test_e4m3_table():
    assert len(O.E4M3) == 127 and O.E4M3[-1] == 448 and O.E4M3[1] == 2.0 ** -9 and O.E4M3[0x38] == 1.0
    assert (np.diff(O.E4M3) > 0).all()
    # a tie between 1 and 1.125 goes to the even code, 1
    assert O.E4M3[O.nearest_code(np.array([1.0625, 1.0626, 1000.0]), O.E4M3)].tolist() == [1.0, 1.125, 448.0]


def test_block_scales_by_hand():
    x = np.zeros((1, 128))
    x[0, 0], x[0, 33], x[0, 64] = 6.0, -0.4, 1.0
    c, b = O.fp4_quantize(x, "e8m0_32")
    # 2^(2 - 2) = 1; 0.4 = 1.6 * 2^-2 -> 2^-4; 2^(0 - 2); a block of zeros 2^-127
    assert b.tolist() == [[127, 123, 125, 0]]
    v = O.fp4_values(c, b, "e8m0_32")
    assert v[0, 0] == 6 and v[0, 33] == -6 * 2.0 ** -4 and v[0, 64] == 1.0
    c, b = O.fp4_quantize(x, "e4m3_16")
    s = O.E4M3[b[0]]
    assert s[0] == 1.0 and s[4] == O.E4M3[O.nearest_code(np.array([1 / 6]), O.E4M3)][0] and s[1] == 0
    assert c[0, 33] == 8 + 7                                        # minus the largest level


@pytest.mark.parametrize("fmt", ["e8m0_32", "e4m3_16"])
def test_quantization_invariants(fmt):
    r = np.random.default_rng(0)
    x = r.normal(size=(200, 256)) * np.exp(r.normal(size=(200, 1)) * 3)
    c, b = O.fp4_quantize(x, fmt)
    v = O.fp4_values(c, b, fmt)
    assert (np.sign(v) * np.sign(x) >= 0).all()
    top = np.abs(x.reshape(200, -1, O.BLOCK[fmt])).max(2).repeat(O.BLOCK[fmt], 1)
    # half the widest step (1 of 6) of the block's scale, plus what saturates: up to a quarter of the largest (8 -> 6).
    # An e4m3 scale is off by up to 2^-10 more below 2^-6 (its subnormal step is 2^-9), which moves a value by at most
    # six times that, and it ends at 448, which cuts values off at 6 * 448.
    tol = 0.26 * top
    if fmt == "e4m3_16":
        tol = tol + 6 * 2.0 ** -10 + np.maximum(np.abs(x) - 6 * 448, 0)
    assert (np.abs(v - x) <= tol).all()
    np.testing.assert_array_equal(O.fp4_quantize(4 * x, fmt, 4.0)[0], c)
    np.testing.assert_array_equal(O.fp4_values(*O.fp4_quantize(-x, fmt), fmt), -v)


def test_tiled_scales_by_hand():
    b = np.arange(130 * 8).reshape(130, 8) % 251
    t = O.tile_scales(b.astype(np.uint8))
    assert t.size == 2 * 2 * 512
    assert t[0] == b[0, 0] and t[3] == b[0, 3] and t[16] == b[1, 0] and t[4] == b[32, 0] and t[512] == b[0, 4]
    assert t[1024 + 16] == b[129, 0] and t[1024 + 32] == 0


def test_route_by_hand():
    l = np.array([[2.0, 1.0, 3.0, 3.0]])
    ids, w, counts = O.route_gated(l, 2)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, 0.5) and counts.tolist() == [0, 0, 1, 1]
    ids, w, _ = O.route_gated(l, 2, score="sigmoid", bias=np.array([1.0, 0, 0, 0]), renormalise=False, scale=2.0)
    assert ids.tolist() == [[0, 2]] and np.allclose(w, 2 / (1 + np.exp([[-2.0, -3.0]])))
    # groups (0, 1) and (2, 3): by the largest the second, by the sum of two the first
    l = np.array([[1.0, 1.0, 2.0, -9.0]])
    assert O.route_gated(l, 1, n_groups=2, group_rank="max")[0].tolist() == [[2]]
    assert O.route_gated(l, 1, score="sigmoid", n_groups=2, group_rank="top2")[0].tolist() == [[0]]


def test_products_and_combination_agree():
    """Combining expert products of segment rows is the dense sum over a token's experts."""
    r = np.random.default_rng(1)
    n, E, k, K, N = 20, 4, 2, 16, 8
    ids, w, counts = O.route_gated(r.normal(size=(n, E)), k)
    starts = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    seg = np.concatenate([starts, counts])
    perm = np.full(starts[-1], -1)
    for e in range(E):
        perm[starts[e]:starts[e] + counts[e]] = np.nonzero((ids == e).any(1))[0]
    x, W = r.normal(size=(n, K)), r.normal(size=(E, N, K))
    z = O.expert_products(np.where(perm[:, None] >= 0, x[perm], 0), W, seg)
    want = np.stack([sum(w[t, j] * (W[ids[t, j]] @ x[t]) for j in range(k)) for t in range(n)])
    np.testing.assert_allclose(O.combine(z, ids, w, seg, perm, E), want, rtol=1e-12)
