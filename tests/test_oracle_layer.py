"""Pins of the float64 restatements around a layer's attention and experts."""
import numpy as np
import pytest

from oracle import kv4 as K
from oracle import layer as Y


def test_e4m3_values():
    assert Y.e4m3(0x7E) == 448 and Y.e4m3(0xFE) == -448 and Y.e4m3(1) == 2.0 ** -9 and Y.e4m3(8) == 2.0 ** -6 and np.isnan(Y.e4m3(0x7F))
    torch = pytest.importorskip("torch")
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Y.e4m3(np.arange(256)), ref, equal_nan=True)


def test_norm_of_a_known_row():
    h, y = Y.add_norm(np.array([[1.0, 2.0]]), np.array([[2.0, 2.0]]), np.array([2.0, 0.5]), 0.0)
    assert h.tolist() == [[3, 4]] and np.allclose(y, [[6 / 12.5 ** 0.5, 2 / 12.5 ** 0.5]])
    assert Y.scales(np.array([[448.0, -2, 896, 1]]), 2).tolist() == [[1, 2]] and Y.scales(np.array([[448.0, -2, 896, 1]]), 0).tolist() == [[2]]


def test_route_by_hand():
    ids, gates = Y.route([[0.0, np.log(3.0), np.log(2.0)]], 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(gates, [[0.5, 1 / 3]])
    ids, gates = Y.route([[0.0, np.log(3.0), np.log(2.0)]], 2, renorm=True, scale=2)
    assert np.allclose(gates, [[1.2, 0.8]])
    # the bias chooses and does not weigh
    ids, gates = Y.route([[0.0, 0.0, 0.0]], 1, sigmoid=True, bias=[0, 0.1, 0.1])
    assert ids.tolist() == [[1]] and np.allclose(gates, 0.5)
    # groups: the second one's best two beat the first one's best
    ids, _ = Y.route([[3.0, -9, 2.5, 2.5]], 2, sigmoid=True, groups=2, top_groups=1, best=2)
    assert ids.tolist() == [[2, 3]]
    ids, _ = Y.route([[3.0, -9, 2.5, 2.5]], 2, sigmoid=True, groups=2, top_groups=1, best=1)
    assert ids.tolist() == [[0, 1]]
    ids, gates = Y.route([[-np.inf] * 3], 2, renorm=True)
    assert ids.tolist() == [[0, 1]] and not gates.any()
    _, gates = Y.route([[-900.0, -901.0]], 2, sigmoid=True, renorm=True)
    assert np.allclose(gates, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]])


def test_bounds_hold_and_are_tight():
    r = np.random.RandomState(0)
    for scale in (1e-6, 1.0, 3e4):
        k = r.randn(13, 64) * scale
        hi, lo, step = Y.bounds(k)
        f = k.astype(np.float32)
        assert (hi * step >= f.max(0)).all() and (lo * step <= f.min(0)).all()
        assert (hi * step - f.max(0) < step).all() and max(abs(hi).max(), abs(lo).max()) >= 64
    assert Y.bounds(np.full((2, 64), 127.0))[2] == 1 and Y.bounds(np.full((2, 64), 127.5))[2] == 2
    assert Y.bounds(np.zeros((2, 64)))[2] == 0


def test_scores_bound_the_products():
    r = np.random.RandomState(1)
    for G in (1, 3, 8):
        k, q = r.randn(16, 64), r.randn(G, 64)
        hi, lo, step = Y.bounds(k)
        up, down = Y.whole_query(q)
        bits = 15 - int(np.ceil(np.log2(G)))
        unit = np.abs(q).max() / 2.0 ** (bits - 1)            # at least q's step
        exact = (k @ q.T).sum(1).max()
        score = step * (hi @ up + lo @ down) * 2.0 ** (np.frexp(np.abs(q).max())[1] - bits)
        assert score >= exact - G * 64 * unit * np.abs(k).max()
        assert np.abs(up).max() < 2 ** 15 and np.abs(down).max() < 2 ** 15


def test_all_blocks_are_plain_attention():
    r = np.random.RandomState(2)
    P, hkv, D, kv, ql = 16, 2, 64, [37, 5], [2, 1]
    pages = np.stack([np.concatenate([K.pack_page(*K.quantise(r.randn(P, D)), *K.quantise(r.randn(P, D))) for _ in range(hkv)]) for _ in range(4)])
    table = np.array([[2, 0, 3], [1, -1, -1]])
    q, qs = r.randn(3, 4, D), np.array([0, 2, 3])
    ks, vs = zip(*[K.unpack(pages, table[b], kv[b], P, hkv, D) for b in range(2)])
    sel = np.tile(np.array([0, 1, 2, -1]), (3, hkv, 1))
    a, sa = Y.attention_blocks(q, qs, kv, table, pages, P, hkv, sel, 0.3)
    b, sb = K.attention(q, qs, list(ks), list(vs), 0.3)
    assert np.allclose(a, b) and np.allclose(sa, sb)


def test_select_lists():
    codes, steps = np.zeros((6, 1, 2, 64), np.int8), np.ones((6, 1))
    codes[:, 0, 0, 0] = [1, 9, 3, 9, 5, 0]
    q = np.zeros((1, 1, 64))
    q[0, 0, 0] = 1.0
    table = np.arange(6)[None]

    def pick(top, first, last, kv=96):
        return Y.select(q, [0, 1], [kv], table, codes, steps, 16, top, first, last, np.full((1, 1, top), -7), 1000)[0, 0].tolist()
    assert pick(3, 1, 1) == [0, 1, 5] and pick(4, 1, 1) == [0, 1, 3, 5] and pick(1, 0, 0) == [1] and pick(2, 0, 0) == [1, 3]
    assert pick(7, 1, 1) == [0, 1, 2, 3, 4, 5, -1] and pick(3, 1, 1, 20) == [0, 1, -1] and pick(2, 0, 2) == [4, 5] and pick(2, 1, 1, 2000) == [-1, -1]
