"""The float64 reference of the router's backward pass against differences of its
own forward definitions, and hand-worked losses."""
import numpy as np
import pytest

import router_train_testlib as ref


def _case(mode, seed, T=7, E=6, k=3):
    rng = np.random.default_rng(seed)
    l = rng.normal(size=(T, E)) * 2
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    seq = np.array([0, 0, 2, -1, 2, 2, 0])[:T]
    return rng, l, idx, seq


@pytest.mark.parametrize("mode,eps", [("sigmoid", 0.0), ("softmax", 1e-8), ("softmax", 0.9)])
def test_gradient_against_differences(mode, eps):
    rng, l, idx, seq = _case(mode, 3)
    n_seq, k = 4, idx.shape[1]
    counts, tokens = ref.counts_of(idx, seq, n_seq, l.shape[1])
    g, gl = rng.normal(size=idx.shape), np.array([0.7, -0.3])
    live = (seq >= 0)[:, None]

    def value(x):
        b, z = ref.losses(x, counts, tokens, seq, mode, k)
        return gl[0] * b + gl[1] * z + (live * g * ref.weights(x, idx, mode, 2.5, eps)).sum()

    d, mag = ref.grad_logits(l, idx, seq, n_seq, mode, scale=2.5, eps=eps, grad_w=g, grad_losses=gl, counts=counts, tokens=tokens)
    assert (np.abs(d) <= mag + 1e-12).all()
    h = 1e-6
    for t in range(l.shape[0]):
        for e in range(l.shape[1]):
            x, y = l.copy(), l.copy()
            x[t, e] += h
            y[t, e] -= h
            assert abs((value(x) - value(y)) / (2 * h) - d[t, e]) < 1e-7


def test_even_loads_and_scores_give_one():
    E, k, T = 4, 2, 8
    idx = np.array([[t % E, (t + 1) % E] for t in range(T)])
    seq = np.zeros(T, int)
    counts, tokens = ref.counts_of(idx, seq, 1, E)
    assert counts.tolist() == [[4, 4, 4, 4]] and tokens.tolist() == [8]
    for mode in ("sigmoid", "softmax"):
        b, z = ref.losses(np.zeros((T, E)), counts, tokens, seq, mode, k)
        assert abs(b - 1) < 1e-15 and abs(z - np.log(4) ** 2) < 1e-15


def test_all_tokens_on_one_expert():
    """One expert with every choice and every score: balance = E."""
    E = 5
    idx, seq = np.full((3, 1), 2), np.zeros(3, int)
    counts, tokens = ref.counts_of(idx, seq, 1, E)
    l = np.full((3, E), -800.0)
    l[:, 2] = 0
    assert abs(ref.losses(l, counts, tokens, seq, "softmax", 1)[0] - E) < 1e-12
