"""Pins of the shaping oracle: closed forms and central differences."""
import numpy as np
import pytest

from oracle import shaping_oracle as so


def test_neutral_row_is_the_row_itself():
    z = np.random.default_rng(0).standard_normal(17)
    zp, slope, _ = so.shape_row(z, history=[3, 3, 5], prompt_len=1)
    assert np.array_equal(zp, z) and np.all(slope == 1.0)


def test_hand_worked_row():
    # history: prompt (2), output (0, 0, 3); theta 2, f 0.25, p 0.5, T 0.5, bias +1 on 3, token 4 barred
    z = np.array([3.0, -1.0, 4.0, -2.0, 9.0])
    zp, slope, _ = so.shape_row(z, [2, 0, 0, 3], 1, 2.0, 0.5, 0.25, [(3, 7.0), (3, 1.0)],
                                np.array([1, 1, 1, 1, 0], bool), 0.5)
    # 0: 3/2 - 2*.25 - .5 = .5; 1: -1; 2: 4/2 = 2; 3: -4 - .25 - .5 + 1 = -3.75
    assert np.array_equal(zp, [1.0, -2.0, 4.0, -7.5, -np.inf])
    assert np.array_equal(slope, [1.0, 2.0, 1.0, 4.0, 0.0])


def test_no_allowed_token():
    zp, _, _ = so.shape_row(np.zeros(3), allowed=np.zeros(3, bool))
    logp, lse = so.shaped_logp(zp[None], [1], [1])
    assert lse[0] == -np.inf and logp[0] == -np.inf
    assert np.all(so.shaped_logp_grad(zp[None], np.zeros((1, 3)), [1], [1], lse, [1.0]) == 0)


def test_uniform_row_closed_form():
    zp, _, _ = so.shape_row(np.zeros(10), allowed=np.arange(10) < 4, temperature=3.0)
    logp, lse = so.shaped_logp(zp[None], [2], [1])
    assert lse[0] == pytest.approx(np.log(4)) and logp[0] == pytest.approx(-np.log(4))


def test_gradient_by_central_differences():
    rng = np.random.default_rng(1)
    n, V = 4, 23
    Z = rng.standard_normal((n, V)) * 2
    batch = dict(tokens=rng.integers(0, V, 20), hist_begin=[0, 3, 0, 11], hist_len=[5, 9, 0, 7],
                 prompt_len=[2, 0, 0, 7], repetition=[1.4, 0.8, 1.2, 1.1], presence=[0.2, 0.0, 0.3, 0.1],
                 frequency=[0.1, 0.4, 0.0, 0.2], temperature=[0.7, 1.0, 1.3, 0.9],
                 bias_offsets=[0, 3], bias_tokens=[1, 4, 8], bias_values=[0.5, -1.0, 2.0], bias_set=[0, -1, 0, -1],
                 allow_bits=rng.integers(0, 1 << 23, (1, 1)).astype(np.uint32).view(np.int32), allow_row=[-1, 0, -1, 0])
    ok = [(int(np.uint32(batch["allow_bits"][0, 0])) >> j) & 1 for j in range(V)]
    y = [3, int(np.argmax(ok)), 7, int(np.argmax(ok))]
    mask, coef = [1, 1, 1, 1], np.array([0.3, -0.7, 1.1, 0.4])

    def loss(Z):
        zp = so.shape_logits(Z, batch)[0]
        return float(np.sum(coef * so.shaped_logp(zp, y, mask)[0]))

    zp, slope, _, bad = so.shape_logits(Z, batch)
    assert not bad.any()
    G = so.shaped_logp_grad(zp, slope, y, mask, so.shaped_logp(zp, y, mask)[1], coef)
    h = 1e-5   # no |z| is below it: the penalty's kink at 0 is not crossed
    assert np.min(np.abs(Z)) > h
    for i in range(n):
        for j in range(V):
            Zp, Zm = Z.copy(), Z.copy()
            Zp[i, j] += h
            Zm[i, j] -= h
            assert (loss(Zp) - loss(Zm)) / (2 * h) == pytest.approx(G[i, j], abs=1e-8)
