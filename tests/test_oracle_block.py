"""Pins of the fp64 definitions in oracle/block.py: gradients against central differences, closed
forms, special cases."""
import numpy as np
import pytest

from oracle import block as K


def _diff(f, x, eps=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        d[i] = (up - f()) / (2 * eps)
        x[i] = keep
    return d


@pytest.mark.parametrize("gate_mode", [0, 1])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 0, 3]])
def test_scan_gradient_is_the_central_difference(gate_mode, tied, lengths):
    rng = np.random.default_rng(3)
    x, g = rng.normal(size=(3, 5, 2)), rng.normal(size=(3, 5, 2))
    g = -np.exp(g) if gate_mode == 0 else g
    h0, dh, dhT = rng.normal(size=(3, 2)), rng.normal(size=(3, 5, 2)), rng.normal(size=(3, 2))

    def loss():
        h, s, _ = K.scan_fwd(x, g, h0, gate_mode, tied, lengths)
        return (h * dh).sum() + (s * dhT).sum()

    for got, at in zip(K.scan_bwd(x, g, h0, dh, dhT, gate_mode, tied, lengths), (x, g, h0)):
        assert np.max(np.abs(got - _diff(loss, at))) < 1e-7      # eps^2 times third derivatives, 1e-16 / eps


def test_scan_closed_forms():
    x = np.ones((1, 40, 1))
    h, s, _ = K.scan_fwd(x, np.full((1, 40, 1), np.log(0.5)), gate_mode=0)
    assert np.allclose(h[0, :, 0], 2 - 0.5 ** np.arange(40.0), rtol=1e-14)      # a geometric sum
    h, _, _ = K.scan_fwd(3 * x, np.zeros((1, 40, 1)), np.full((1, 1), 3.0), tied=True)
    assert np.allclose(h, 3.0, rtol=1e-15)                       # an average of equal values
    h, s, _ = K.scan_fwd(x, np.full((1, 40, 1), 800.0))          # the gate shuts: nothing is kept
    assert np.all(h == 1.0)


def test_layernorm_gradient_is_the_central_difference():
    rng = np.random.default_rng(4)
    x, w, b, dy = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=5), rng.normal(size=(3, 5))
    loss = lambda: (K.layernorm_fwd(x, w, b)[0] * dy).sum()
    for got, at in zip(K.layernorm_bwd(x, dy, w), (x, w, b)):
        assert np.max(np.abs(got - _diff(loss, at))) < 1e-7


def test_beam_select_by_hand():
    logits = np.log(np.array([[[0.5, 0.25, 0.25], [0.9, 0.1, 0.0 + 1e-300]]]))
    s, p, t = K.beam_select(logits, np.log([[0.6, 0.4]]), 4)
    assert p.tolist() == [[1, 0, 0, 0]] and t.tolist() == [[0, 0, 1, 2]]        # 0.36, 0.30, 0.15, 0.15
    assert np.allclose(np.exp(s), [[0.36, 0.30, 0.15, 0.15]])
    # a finished beam keeps its score as one candidate, an empty one has none; -inf fills by index
    s, p, t = K.beam_select(np.zeros((1, 3, 2)), np.array([[-1.0, -np.inf, -0.5]]), 5, np.array([[True, False, False]]), 1)
    assert p[0].tolist() == [0, 2, 2, 0, 1] and t[0].tolist() == [1, 0, 1, 0, 0]
    assert np.all(s[0, 3:] == -np.inf)


def test_a_poisoned_beam_drops_out():
    logits = np.zeros((1, 4, 3))
    logits[0, 0, 1] = np.nan
    logits[0, 1, 2] = np.inf
    logits[0, 2] = -np.inf
    s, p, t = K.beam_select(logits, np.zeros((1, 4)), 4)
    assert p[0].tolist() == [3, 3, 3, 0] and t[0].tolist() == [0, 1, 2, 0]


def test_state_reorder_reads_before_it_writes():
    S = np.arange(6.0).reshape(6, 1)
    out = K.state_reorder(S, np.array([[1, 0, 0], [2, 2, 7]]))
    assert out[:, 0].tolist() == [1, 0, 0, 5, 5, 5]
