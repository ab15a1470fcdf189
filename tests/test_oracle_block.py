"""Pins of the oracle of the operators around the expert layer (CPU): closed forms and finite
differences of every gradient."""
import numpy as np
import pytest

from oracle import block_ref as R
from oracle import moe_ref


def test_norm_closed_forms():
    h = np.array([[3.0, -4.0], [0.0, 0.0]])
    y, r = R.rms_norm(h, np.array([1.0, 2.0]), 0.5)
    np.testing.assert_allclose(y[0], [3 / np.sqrt(13.0), -8 / np.sqrt(13.0)], rtol=1e-15)
    assert (y[1] == 0).all() and r[1, 0] == pytest.approx(2 ** 0.5)


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(0)
    h, w, dy, res = (rng.standard_normal(s) for s in ((3, 8), 8, (3, 8), (3, 8)))
    dh, dw = R.rms_norm_bwd(dy, h, w, 1e-3, res)
    f = lambda h, w: (R.rms_norm(h, w, 1e-3)[0] * dy).sum() + (h * res).sum()  # noqa: E731
    for i in np.ndindex(3, 8):
        e = np.zeros_like(h)
        e[i] = 1e-5
        assert (f(h + e, w) - f(h - e, w)) / 2e-5 == pytest.approx(dh[i], abs=1e-8)
    for j in range(8):
        e = np.zeros(8)
        e[j] = 1e-5
        assert (f(h, w + e) - f(h, w - e)) / 2e-5 == pytest.approx(dw[j], abs=1e-8)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_balance_gradient_by_differences(sigmoid):
    rng = np.random.default_rng(1)
    T, E, k = 9, 6, 2
    x = rng.standard_normal((T, E))
    idx = np.argsort(-x, 1)[:, :k]
    off, mask = [1, 4, 4, 8], np.array([1, 1, 0, 1, 1, 1, 1, 1, 1])
    got = R.seq_aux(x, idx, off, mask, sigmoid, 0.7, 0.3)
    assert got["tokens"].tolist() == [2, 0, 4]
    for i in np.ndindex(T, E):
        e = np.zeros_like(x)
        e[i] = 1e-5
        d = (R.seq_aux(x + e, idx, off, mask, sigmoid, 0.7, 0.3)["loss"].sum()
             - R.seq_aux(x - e, idx, off, mask, sigmoid, 0.7, 0.3)["loss"].sum()) / 2e-5
        assert d == pytest.approx(got["d_logits"][i], abs=1e-8)
    assert (got["d_logits"][[0, 2, 8]] == 0).all()


@pytest.mark.parametrize("sigmoid", [0, 1])
def test_one_sequence_is_the_whole_batchs_loss(sigmoid):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((12, 5)).astype(np.float32)
    idx = np.argsort(-x, 1)[:, :2].astype(np.int32)
    got = R.seq_aux(x, idx, [0, 12], None, bool(sigmoid), 0.25, 0.0)
    loss, counts, probs = moe_ref.aux_loss(x, idx, 5, sigmoid, 0.25)
    assert (got["counts"][0] == counts).all()
    np.testing.assert_allclose(got["probs"][0], probs, rtol=1e-12)
    assert got["loss"][0] == pytest.approx(float(loss), rel=1e-12)


def test_rows_without_a_logit_add_nothing():
    x = np.full((2, 3), -np.inf)
    x[0] = [0.0, 0.0, -np.inf]
    got = R.seq_aux(x, np.array([[0], [1]]), [0, 2], None, False, 1.0, 1.0)
    np.testing.assert_allclose(got["probs"][0], [0.25, 0.25, 0.0])
    assert got["loss"][1] == pytest.approx(np.log(2.0) ** 2 / 2) and (got["d_logits"][1] == 0).all()


def test_vanishing_scores_keep_their_proportions():
    """Sigmoids of far negative logits are e^x: their quotients are the softmax; of equal ones 1 / E."""
    x = np.array([[-900.0, -901.0, -np.inf], [-1e30, -1e30, -1e30]])
    p, jac, soft, _ = R.probabilities(x, True)
    np.testing.assert_allclose(p, soft, rtol=1e-12)
    np.testing.assert_allclose(jac, p, rtol=1e-12)
    np.testing.assert_allclose(p[1], 1 / 3)
    x = np.array([[800.0, -2.0]])
    p, jac, _, _ = R.probabilities(x, True)
    s = 1 / (1 + np.exp(2.0))
    np.testing.assert_allclose(p, [[1 / (1 + s), s / (1 + s)]], rtol=1e-12)
    np.testing.assert_allclose(jac, [[0.0, s * (1 - s) / (1 + s)]], rtol=1e-12, atol=1e-300)


def test_clip_closed_forms():
    g = [np.array([3.0]), np.array([0.0, 4.0])]
    norm, c = R.clip(g, 1.0, 0.5)
    assert norm == 2.5 and c == pytest.approx(0.2, rel=1e-6)
    assert R.clip(g, 10.0, 0.5) == (2.5, 0.5)
    assert R.clip([np.array([np.inf])], 1.0, 0.5) == (np.inf, 0.5)
