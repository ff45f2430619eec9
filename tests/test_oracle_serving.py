"""Pins of the oracle's serving operators: the grouped product of packed layers
and the log probabilities of given tokens."""
import numpy as np
import pytest

from oracle import slim_oracle as O


def layers(E, m, n, group, avg, seed):
    rng = np.random.default_rng(seed)
    k = n // group
    bits = np.stack([O.allocation(rng.permutation(k), avg, k // 3) for _ in range(E)]).astype(np.uint8)
    codes = [np.concatenate([rng.integers(0, 2 ** int(b), (m, group)) for b in bits[e]], axis=1) for e in range(E)]
    words = np.stack([O.pack_codes(codes[e], bits[e], group, avg) for e in range(E)])
    return words, bits, rng.uniform(0.01, 0.02, (E, m, k)), rng.uniform(0, 3, (E, m, k)), codes


def test_grouped_product_by_hand():
    words, bits, scale, zero, codes = layers(3, 4, 96, 32, 2, 0)
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 96))
    offsets, index = [0, 2, 2, 6], [4, 0, 0, 9, 3, -1, 2]
    y = O.dequant_grouped_matmul(words, bits, scale, zero, 32, x, offsets, index)
    for r, (e, src) in enumerate([(0, 4), (0, 0), (2, 0), (2, 9), (2, 3), (2, -1)]):
        for i in range(4):
            want = 0.0
            for j in range(96):
                xv = x[src, j] if 0 <= src < 5 else 0.0
                want += xv * scale[e, i, j // 32] * (codes[e][i, j] - zero[e, i, j // 32])
            assert abs(y[r, i] - want) < 1e-12
    assert np.isnan(y[6]).all()


def test_token_logprobs_closed_forms():
    # uniform over 8: logp = -log 8, entropy log 8, ties rank by index
    logp, ent, tl, ti = O.token_logprobs(np.zeros((1, 8)), [5], 3)
    assert np.allclose([logp[0], ent[0]], [-np.log(8), np.log(8)]) and ti.tolist() == [[0, 1, 2]]
    assert np.allclose(tl, -np.log(8))
    # two outcomes with odds 3:1, the rest masked
    l = np.array([[-np.inf, np.log(3.0), -np.inf, 0.0]])
    logp, ent, tl, ti = O.token_logprobs(l, [0], 4)
    assert np.isneginf(logp[0]) and np.allclose(ent, np.log(4) - 0.75 * np.log(3))
    assert ti.tolist() == [[1, 3, 0, 2]] and np.allclose(tl[0, :2], np.log([0.75, 0.25])) and np.isneginf(tl[0, 2:]).all()
    # nothing left
    logp, ent, tl, ti = O.token_logprobs(np.full((1, 4), -np.inf), [1], 2)
    assert np.isneginf(logp[0]) and ent[0] == 0 and np.isneginf(tl).all() and ti.tolist() == [[0, 1]]
    # no token, a huge offset, NaN
    assert O.token_logprobs(np.zeros((2, 3)), [-100, 3])[0].tolist() == [0, 0]
    assert np.allclose(O.token_logprobs(np.array([[1e30, 1e30]]))[1], np.log(2))
    logp, ent, tl, ti = O.token_logprobs(np.array([[0.0, np.inf, np.nan, 1.0]]), [0], 2)
    assert np.isnan([logp[0], ent[0], *tl[0]]).all() and ti.tolist() == [[2, 1]]
    assert np.isnan(O.token_logprobs(np.array([[0.0, np.inf]]), [0])[0][0])


@pytest.mark.parametrize("seed", [0, 1])
def test_entropy_is_minus_expected_logp(seed):
    l = np.random.default_rng(seed).standard_normal((4, 50)) * 4
    lp = np.stack([O.token_logprobs(l, np.full(4, v))[0] for v in range(50)], axis=1)
    assert np.allclose(np.exp(lp).sum(1), 1) and np.allclose(O.token_logprobs(l)[1], -(np.exp(lp) * lp).sum(1))
