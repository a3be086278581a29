"""Pins of the paged oracle: hand-worked pages, a rotation known in closed
form, and the attention against the dense oracle; each pin fails for a
planted mistake."""
import numpy as np
import pytest

import oracle.diffattn_ref as ref
import oracle.paged_ref as pr


def test_step_by_hand():
    # pages of 4; request 0 goes 3 -> 5 (takes one), 1 is finished (returns two), 2 goes 8 -> 9 (takes one)
    table = np.array([[7, -1, -1], [2, 5, -1], [1, 3, -1]])
    ring = np.array([9, 6, 0, -1, -1, 8])
    got = pr.paged_step([3, 6, 8], [2, -1, 1], table, ring, [5, 4], 4, 5)
    t, r, pool, cu, kv, pos, slots, info = got
    assert t.tolist() == [[7, 8, -1], [2, 5, -1], [1, 3, 9]]
    assert r.tolist() == [9, 6, 0, 2, 5, 8]  # ring slots 3 and 4: behind the four live ones at 5, 0, 1, 2
    assert pool == [1, 4] and cu == [0, 2, 2, 3] and kv == [5, 0, 9]
    assert pos == [3, 4, 8, -1, -1] and slots == [7 * 4 + 3, 8 * 4, 9 * 4, -1, -1]
    assert info == [3, 2, 2, 0]


def test_step_refusals_by_hand():
    table, ring = np.full((2, 2), -1), np.array([0, 1, 2])
    code = lambda ctx, new, pool=(0, 3), T=50: pr.paged_step(ctx, new, table, ring, pool, 4, T)[7][3]
    assert code([0, 0], [8, 4]) == 0
    assert code([0, 0], [8, 8]) == 1
    assert code([0, 0], [9, 0]) == 2
    assert code([0, 0], [8, 4], T=11) == 4
    assert code([0, 0], [-2, 4]) == 8
    assert code([0, 0], [4, 0], pool=(3, 2)) == 16


def test_rotation_in_closed_form():
    x = np.array([[[1.0, 0.0, 1.0, 0.0, 5.0]]])
    y = pr.rope(x, np.array([1]), np.array([np.pi / 2, np.pi]), half=False)
    assert np.allclose(y, [[[0, 1, -1, 0, 5]]], atol=1e-15)
    y = pr.rope(x, np.array([1]), np.array([np.pi / 2, np.pi]), half=True)  # pairs (0, 2), (1, 3)
    assert np.allclose(y, [[[-1, 0, 1, 0, 5]]], atol=1e-15)
    th, m = pr.rope_frequencies(8, 1e4, "yarn", 8.0)
    assert np.allclose(pr.rope(pr.rope(x[..., :4], np.array([9]), th[:2], m), np.array([9]), th[:2], 1 / m,
                               inverse=True), x[..., :4])


def test_scaled_frequencies():
    plain = 1e4 ** (-np.arange(0, 128, 2) / 128)
    assert np.allclose(pr.rope_frequencies(128, 1e4)[0], plain)
    assert np.allclose(pr.rope_frequencies(128, 1e4, "linear", 4.0)[0], plain / 4)
    ntk = pr.rope_frequencies(128, 1e4, "ntk", 4.0)[0]
    assert np.isclose(ntk[0], 1) and np.isclose(ntk[-1], plain[-1] / 4)  # the slowest pair is interpolated fully
    th, m = pr.rope_frequencies(128, 1e4, "yarn", 4.0)
    assert np.isclose(m, 1 + 0.1 * np.log(4)) and np.isclose(th[0], 1) and np.isclose(th[-1], plain[-1] / 4)


def _dense(seed, n, H, d):
    r = np.random.default_rng(seed)
    return r.standard_normal((1, n, H, 2, d)), r.standard_normal((1, n, H, 2, d)), r.standard_normal((1, n, H, 2 * d))


@pytest.mark.parametrize("causal", [True, False])
def test_extend_against_the_dense_oracle(causal):
    n, H, d, page = 11, 2, 4, 4
    q, k, v = _dense(1, n, H, d)
    w, lam = np.linspace(0.5, 1.5, 2 * d), 0.4
    want = ref.diffattn_fwd(q, k, v, lam, 0.3, w, 1e-5, causal)[0]
    ids = np.array([4, 0, 2])
    kc, vc = np.full((5, page, H, 2, d), np.nan), np.full((5, page, H, 2 * d), np.nan)
    for i in range(n):
        kc[ids[i // page], i % page], vc[ids[i // page], i % page] = k[0, i], v[0, i]
    new = 6 if causal else n
    got = pr.extend(q[0, n - new:], kc, vc, ids[None], [0, new], [n], lam, 0.3, w, 1e-5, causal)
    assert np.allclose(got, want[n - new:], atol=1e-12)


def test_extend_shared_heads_and_empty_rows():
    n, d = 5, 4
    q, k, v = _dense(2, n, 3, d)
    w = np.ones(2 * d)
    kc, vc = k[0][None], v[0][None]  # one page of 5
    own = pr.extend(q[0], kc[:, :, :1], vc[:, :, :1], np.array([[0]]), [0, n], [n], 0.4, 0.3, w, 1e-5)
    rep = pr.extend(q[0], kc[:, :, [0, 0, 0]], vc[:, :, [0, 0, 0]], np.array([[0]]), [0, n], [n], 0.4, 0.3, w, 1e-5)
    assert np.array_equal(own, rep)
    short = pr.extend(q[0], kc, vc, np.array([[0]]), [0, n], [3], 0.4, 0.3, w, 1e-5)
    assert (short[:2] == 0).all() and np.abs(short[2:]).min() > 0
