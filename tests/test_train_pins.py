"""Pins of the training step's oracle (oracle/train.py): hand-worked values,
masked and empty cases, gradients against differences."""
import numpy as np
import pytest

from oracle import train as R

INF = float("inf")


def test_balance_by_hand():
    # two tokens, p = (1/4, 3/4) and (1/2, 1/2); both choose expert 1
    x = np.log([[1.0, 3.0], [1.0, 1.0]])
    loss, counts, prob = R.balance(x, [[1], [1]])
    assert counts.tolist() == [[0, 2]] and np.allclose(prob, [[0.375, 0.625]])
    assert np.allclose(loss, [2 / 2 * 2 * 0.625])
    # an even choice of even scores costs 1, whatever k
    loss, _, _ = R.balance(np.zeros((4, 4)), [[0, 1], [2, 3], [0, 1], [3, 2]])
    assert np.allclose(loss, [1.0])


def test_balance_sequences_and_masks():
    x = np.array([[0.0, -INF], [-INF, -INF], [0.0, 0.0], [9.0, 9.0]])
    ids = [[0], [-1], [1], [0]]
    loss, counts, prob = R.balance(x, ids, [0, 2, 2, 3])
    assert counts.tolist() == [[1, 0], [0, 0], [0, 1]]
    assert np.allclose(prob, [[0.5, 0], [0, 0], [0.5, 0.5]])
    assert np.allclose(loss, [2 / 2 * 0.5, 0, 2 * 0.5])
    p = R.scores(np.array([0.0, np.log(3.0), -INF]), "sigmoid")
    assert np.allclose(p, [0.4, 0.6, 0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(4)
    T, E, k = 7, 5, 2
    x = rng.normal(size=(T, E))
    x[2, 3] = -INF
    ids = np.argsort(-x, 1)[:, :k]
    off, dloss = [1, 4, 4, 6], rng.normal(size=3)
    loss, counts, _ = R.balance(x, ids, off, score)
    d, _ = R.balance_backward(x, counts, dloss, k, off, score)
    assert np.all(d[[0, 6]] == 0) and d[2, 3] == 0
    for t in range(T):
        for e in range(E):
            if np.isinf(x[t, e]):
                continue
            v = [x.copy(), x.copy()]
            v[0][t, e] += 1e-5
            v[1][t, e] -= 1e-5
            up, down = (float(dloss @ R.balance(u, ids, off, score)[0]) for u in v)
            assert abs((up - down) / 2e-5 - d[t, e]) < 1e-8


def test_pack_by_hand():
    x = np.zeros((1, 70))
    x[0, 0], x[0, 1], x[0, 2] = 127.0, 0.5, 1.5          # step 1, ties to even
    x[0, 32], x[0, 33] = 127.5, -1.0                     # just past: step 2
    x[0, 64] = 2.0 ** -140                               # below the least step
    q, s = R.pack(x)
    assert s.tolist() == [[127, 128, 1]]
    assert q[0, :3].tolist() == [127, 0, 2] and q[0, 32:34].tolist() == [64, 0]
    assert not q[0, 64:].any()
    v = R.unpack(q, s)
    assert v[0, 0] == 127 and v[0, 32] == 128 and v[0, 64] == 0
    x[0, 40], x[0, 65] = INF, np.nan
    q, s = R.pack(x)
    assert s.tolist() == [[127, 255, 255]] and not q[0, 32:].any()
    assert np.isnan(R.unpack(q, s)[0, 32:]).all()


def test_pack_is_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(20, 96)) * np.exp2(rng.integers(-140, 120, size=(20, 1)))
    q, s = R.pack(x)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, 1)
    assert np.all(np.abs(R.unpack(q, s) - x) <= step / 2)
    # and the step is the least that reaches the block's largest magnitude
    top = np.abs(x).reshape(20, 3, 32).max(2)
    least = np.ldexp(1.0, s.astype(int) - 127)
    assert np.all(top <= 127 * least)
    assert np.all((top > 127 * least / 2) | (s == 1))


def test_gated_gradient_against_differences():
    rng = np.random.default_rng(2)
    gu, dh = rng.normal(size=(3, 10)) * 3, rng.normal(size=(3, 5))
    d, h = R.gated_backward(gu[:, :5], gu[:, 5:], dh)
    assert np.allclose(h, R.gated(gu))
    for i in range(3):
        for j in range(10):
            v = [gu.copy(), gu.copy()]
            v[0][i, j] += 1e-5
            v[1][i, j] -= 1e-5
            up, down = ((dh * R.gated(u)).sum() for u in v)
            assert abs((up - down) / 2e-5 - d[i, j]) < 1e-7
    assert R.gated([[0.0, 5.0]])[0, 0] == 0
    assert R.gated_backward([[0.0]], [[4.0]], [[1.0]])[0].tolist() == [[2.0, 0.0]]


def test_weight_grad_by_hand():
    dy, x = np.array([[1.0, 2.0], [3.0, 0.0], [5.0, 1.0]]), np.array([[1.0], [10.0]])
    out, size = R.weight_grad(dy, x, [0, 2, 2, 3], [2, 1, -4], 2)
    assert out[:, :, 0].tolist() == [[1 * 10 + 3 * 1, 20.0], [0, 0], [0, 0]]
    assert np.array_equal(out, size)
    assert R.weight_grad(dy[:2], x)[0][0, :, 0].tolist() == [31.0, 2.0]


def test_combine_by_hand():
    y = np.array([[1.0, 2.0], [10.0, 20.0]])
    inv, w = [[1, 0], [-1, 2]], [[2.0, 3.0], [5.0, 7.0]]
    out, _ = R.combine(y, inv, w, [[100.0, 0.0], [7.0, 8.0]])
    assert out.tolist() == [[123.0, 46.0], [7.0, 8.0]]
    dy, dw, _ = R.combine_backward([[1.0, -1.0], [4.0, 4.0]], y, inv, w)
    assert dy.tolist() == [[3.0, -3.0], [2.0, -2.0]]
    assert dw.tolist() == [[-10.0, -1.0], [0.0, 0.0]]
    # the gradient is the transpose: <dout, combine(y)> = <combine'(dout), y>
    rng = np.random.default_rng(3)
    inv = rng.permutation(12).reshape(4, 3)
    y, w, d = rng.normal(size=(12, 5)), rng.normal(size=(4, 3)), rng.normal(size=(4, 5))
    dy, dw, _ = R.combine_backward(d, y, inv, w)
    assert np.isclose((dy * y).sum(), (d * R.combine(y, inv, w)[0]).sum())
    assert np.isclose((dw * w).sum(), (d * R.combine(y, inv, w)[0]).sum())
