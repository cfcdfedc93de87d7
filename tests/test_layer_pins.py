"""Pins of the layer oracle (oracle/layer.py): hand-worked values, the masked
and non-finite cases, and the gate's gradient against differences."""
import numpy as np
import pytest

from oracle import layer as L

INF = float("inf")


def test_gate_by_hand():
    # softmax of (0, ln 2, ln 3, ln 2): p = 1/8, 2/8, 3/8, 2/8
    row = np.log([[1.0, 2.0, 3.0, 2.0]])
    ids, w = L.gate(row, 3, renorm=False, scale=2.0)
    assert ids.tolist() == [[2, 1, 3]]          # the tie goes to id 1
    assert np.allclose(w, [[0.75, 0.5, 0.5]], rtol=1e-14)
    ids, w = L.gate(row, 3, renorm=True)
    assert np.allclose(w, [[3 / 7, 2 / 7, 2 / 7]], rtol=1e-14)


def test_gate_sigmoid_by_hand():
    # p = 1/2, 3/4, 1/4; the bias lifts expert 2 over expert 0
    row = np.array([[0.0, np.log(3.0), -np.log(3.0)]])
    ids, w = L.gate(row, 2, "sigmoid", bias=[0.0, 0.0, 0.5], renorm=False)
    assert ids.tolist() == [[1, 2]] or ids.tolist() == [[2, 1]]
    assert np.allclose(sorted(w[0]), [0.25, 0.75], rtol=1e-14)
    ids, w = L.gate(row, 2, "sigmoid", bias=[0.0, 0.0, 0.6], renorm=True)
    assert ids.tolist() == [[2, 1]]
    assert np.allclose(w, [[0.25, 0.75]], rtol=1e-14)


def test_gate_masked_rows():
    rows = np.array([[-INF, 1.0, -INF], [-INF] * 3, [np.nan, 1.0, 2.0],
                     [INF, 0.0, INF]])
    ids, w = L.gate(rows, 2)
    assert ids.tolist() == [[1, -1], [-1, -1], [2, 1], [0, 2]]
    assert w[0].tolist() == [1.0, 0.0] and w[1].tolist() == [0.0, 0.0]
    assert np.isnan(w[2]).all()
    assert w[3].tolist() == [0.5, 0.5]
    low = np.full((1, 4), np.finfo(np.float32).min)
    ids, w = L.gate(low, 2, renorm=False)      # the lowest value is no mask
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.25, 0.25]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(5, 9))
    x[1, 4] = -INF
    x[2, 1:] = -INF
    dw = rng.normal(size=(5, 3))
    ids, _ = L.gate(x, 3, score, renorm=renorm, scale=1.7)
    got = L.gate_backward(x, ids, dw, score, renorm, 1.7)

    def loss(v):
        # weights of the fixed choice, in its order
        total = 0.0
        for t in range(5):
            p = L._row_scores(v[t], score)
            sel = [e for e in ids[t] if e >= 0]
            pw = p[sel] / (p[sel].sum() + 1e-20) if renorm else p[sel]
            total += 1.7 * (pw * dw[t][:len(sel)]).sum()
        return total

    h = 1e-5
    for t in range(5):
        for e in range(9):
            if np.isinf(x[t, e]):
                assert got[t, e] == 0
                continue
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central differences: error h^2 / 6 times a third derivative of
            # order |dw| scale < 10, plus rounding 1e-16 / h
            assert abs((loss(up) - loss(dn)) / (2 * h) - got[t, e]) < 1e-8


def test_quantize_by_hand():
    q, s = L.quantize([[2.0, -1.0, 0.5], [0, 0, 0], [1, INF, 0], [1, np.nan, 0]])
    assert q[0].tolist() == [127, -64, 32]      # 63.5 and 31.75, to even
    assert s[0] == np.float32(2) / np.float32(127)
    assert q[1:].tolist() == [[0, 0, 0]] * 3
    assert s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3])
    q, s = L.quantize(np.full((1, 2), 1e-45, np.float32))
    assert q.tolist() == [[0, 0]] and s[0] == 0


def test_matmul_by_hand():
    a = [[1, -2], [3, 4]]
    w = [[[5, 6], [-7, 8]], [[1, 0], [0, 1]]]
    ws = [[1.0, 0.5], [2.0, 1.0]]
    out = L.matmul_i8(a, [1.0, 10.0], w, ws, offsets=[0, 2, 3, 3, 5],
                      expert_of=[1, 0, 0, 7], index=[3, 0, 2, 1, 1],
                      index_div=2)
    # rows 1, 0 through matrix 1; row 1 through matrix 0; the rest untouched
    assert out[0].tolist() == [60.0, 40.0] and out[1].tolist() == [2.0, -2.0]
    assert out[2].tolist() == [390.0, 55.0] and np.isnan(out[3:]).all()
    out = L.matmul_i8(a, [1.0, 1.0], w[1], ws[1], index=[-1, 0, 9])
    assert out[0].tolist() == [0, 0] and out[2].tolist() == [0, 0]
    assert out[1].tolist() == [2.0, -2.0]
    g = L.matmul_i8([[1, 2]], [1.0], w[1], ws[1], gated=True)
    assert np.allclose(g, 2 / (1 + np.exp(-2.0)) * 2, rtol=1e-14)


def test_moe_by_hand():
    # one token, two experts with weights 3/4 and 1/4, identity-like matrices
    x = np.array([[1.0, 0.0]])
    router = np.array([[np.log(3.0), 0.0], [0.0, 0.0], [-5.0, 0.0]])
    gu = np.zeros((3, 2, 2))
    gu[0] = [[2.0, 0.0], [3.0, 0.0]]
    gu[1] = [[1.0, 0.0], [1.0, 0.0]]
    down = np.array([[[1.0], [0.0]], [[0.0], [1.0]], [[9.0], [9.0]]])
    out, ids, w = L.moe(x, router, gu, down, 2)
    assert ids.tolist() == [[0, 1]]
    assert np.allclose(w, [[0.75, 0.25]], rtol=1e-14)
    s = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    assert np.allclose(out, [[0.75 * s(2) * 3, 0.25 * s(1)]], rtol=1e-14)
