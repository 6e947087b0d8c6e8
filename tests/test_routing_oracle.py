"""Pins of the routing, gradient and int8 oracles (CPU): hand-worked rows, the
gradient against central differences of the weights, and hand-worked codes."""
import numpy as np
import pytest

from oracle import routing

INF = np.inf


def test_gate_hand_worked_rows():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0], [1.0, 1.0, 1.0, 1.0]]))
    ids, w, bad = routing.moe_gate(l, 2)
    assert ids.tolist() == [[1, 2], [0, 1]] and not bad.any()
    assert np.allclose(w, [[0.5, 0.25], [0.25, 0.25]])
    _, w, _ = routing.moe_gate(l, 2, renormalize=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0], [1.5, 1.5]])
    # a bias moves the choice and not the weights
    ids, w, _ = routing.moe_gate(l, 2, bias=np.array([0.0, 0.0, 0.0, 0.9]))
    assert ids.tolist() == [[3, 1], [3, 0]] and np.allclose(w, [[0.125, 0.5], [0.25, 0.25]])


def test_gate_groups_and_masks():
    l = np.array([[3.0, -9.0, 2.0, 2.0, 2.5, -INF]])
    pick = lambda **k: routing.moe_gate(l, 2, score="sigmoid", n_group=3, **k)[0].tolist()
    assert pick(topk_group=1, group_top=1) == [[0, 1]]              # by the best expert
    assert pick(topk_group=1, group_top=2) == [[2, 3]]              # by the sum of two
    assert pick(topk_group=2, group_top=2) == [[0, 2]]
    ids, w, bad = routing.moe_gate(np.array([[-INF, -INF], [0.0, -INF], [np.nan, 0.0], [INF, 0.0]]), 2)
    assert ids.tolist() == [[-1, -1], [0, -1], [-1, -1], [-1, -1]]
    assert w[1].tolist() == [1.0, 0.0] and bad.tolist() == [False, False, True, True]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_central_differences(score, renormalize):
    rng = np.random.default_rng(1)
    T, E, k = 3, 7, 3
    l = rng.standard_normal((T, E))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[1, 2] = -1
    g = rng.standard_normal((T, k))
    d, size = routing.moe_gate_backward(l, ids, g, score, renormalize, 2.5)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            f = lambda x: (routing.chosen_weights(x, ids, score, renormalize, 2.5) * g).sum()
            # central difference: error h^2/6 of a third derivative below 10, and 1e-16/h of rounding
            assert abs((f(up) - f(down)) / (2 * h) - d[t, e]) < 1e-9
    assert (np.abs(d) <= size + 1e-15).all()


def test_tiny_scores_keep_their_ratio():
    l = np.array([[-800.0, -801.0]])
    _, w, _ = routing.moe_gate(l, 2, score="sigmoid", renormalize=True)
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]])


def test_quantize_hand_worked():
    q, s = routing.quantize_int8_per_token(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [np.nan, 1, 2, 3],
                                                     [2.0 ** -130, 0, 0, 0]], np.float32))
    assert q.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0], [0, 0, 0, 0], [0, 0, 0, 0]]   # ties to even
    assert s[0] == 1 and s[1] == 1 and np.isnan(s[2]) and s[3] == np.float32(2.0 ** -126)


def test_codes_are_within_half_a_step():
    """x is within scale / 2 of code * scale: the scale and the inverse are off by half a
    step (2^-24) each, which on 127 codes is 127 * 2.01 * 2^-24 of a scale more."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((200, 64)) * np.exp(rng.uniform(-85, 80, (200, 1)))
    x[:20] = rng.integers(-3, 4, (20, 64)) * 2.0 ** -140          # below the smallest scale
    x[20:40] = rng.integers(-254, 255, (20, 64)) / 2              # halves: ties
    x = x.astype(np.float32)
    q, s = routing.quantize_int8_per_token(x)
    off = np.abs(x.astype(np.float64) - q * s.astype(np.float64)[:, None])
    assert (off <= (0.5 + 256 * 2.0 ** -24) * s[:, None]).all()
    assert (np.abs(q).max(axis=1)[40:] == 127).all() and np.isfinite(s).all()


def test_int8_gemm_hand_worked():
    d = routing.int8_gemm(np.array([[1, -2], [-128, 127]], np.int8), np.array([0.5, 2.0], np.float32),
                          np.array([[3, 4], [-128, -128]], np.int8), np.array([1.0, 0.25], np.float32))
    assert d.tolist() == [[-2.5, 16.0], [2 * (-384 + 508), 0.5 * 128]]
