"""Pins of the 4-bit cache oracle: hand-computed values and properties."""
import numpy as np
import pytest

from oracle import kv4 as K


def test_quantise_hand_values():
    u, s, z = K.quantise(np.array([[0.0, 15.0, 7.0, 7.5, 8.5, 1.0, 2.0, 3.0]]))
    assert s[0] == 1 and z[0] == 0
    assert u[0].tolist() == [0, 15, 7, 8, 8, 1, 2, 3]          # ties to even
    u, s, z = K.quantise(np.full((1, 8), -2.5))
    assert s[0] == 0 and z[0] == -2.5 and not u.any()


def test_quantise_stays_finite():
    x = np.array([[np.inf, -np.inf, np.nan, 1e30, -1e30, 0, 1, 2.0]])
    u, s, z = K.quantise(x)
    assert np.isfinite(s).all() and z[0] == -32768 and u[0, 0] == 15 and u[0, 1] == 0
    assert abs(K.dequantise(u, s, z)[0, 2]) <= float(s[0]) / 2     # NaN is read as 0


def test_quantise_error_is_half_a_step():
    x = np.random.RandomState(0).randn(200, 64)
    u, s, z = K.quantise(x)
    err = np.abs(K.dequantise(u, s, z) - x).max(-1)
    # half a step, the rounding of z (it moves the grid's start) and that of s (15 times at the far end)
    bound = s.astype(float) / 2 + np.abs(z.astype(float)) * 2.0 ** -11 + 15 * s.astype(float) * 2.0 ** -11
    assert (err <= bound).all()


def test_word_layout():
    u = np.zeros((16, 64), np.uint8)
    u[0, :8] = [1, 2, 3, 4, 5, 6, 7, 8]
    one = np.ones(16, np.float16)
    raw = K.pack_page(u, one, one * 0, u, one, one * 0)
    assert raw[:4].view(np.uint32)[0] == 0x86427531
    k, v = K.unpack_head(raw, 16, 64)
    assert np.array_equal(k, u) and np.array_equal(v, u)


def test_bf16_round():
    assert K.bf16_round(np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -7])).tolist() == [1.0, 1.0, 1 + 2.0 ** -6, -1 - 2.0 ** -7]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_relative_positions(interleaved):
    r = np.random.RandomState(1)
    ang = np.arange(50)[:, None] * (0.3 ** np.arange(8))[None]
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = r.randn(1, 1, 16), r.randn(1, 1, 16)

    def dot(i, j):
        a = K.norm_rope(q, None, 0, cs, np.array([i]), interleaved)
        b = K.norm_rope(k, None, 0, cs, np.array([j]), interleaved)
        return float((a * b).sum())
    assert np.isclose(dot(3, 10), dot(33, 40)) and not np.isclose(dot(3, 10), dot(3, 11))


def test_attention_hand_values():
    q = np.ones((2, 1, 2))
    k, v = np.zeros((1, 3, 2)), np.array([[[1.0, 0], [3, 0], [8, 6]]])
    out, _ = K.attention(q, [0, 2], [k], [v], 1.0)
    assert np.allclose(out[:, 0], [[2, 0], [4, 2]])
    out, _ = K.attention(q, [0, 2], [k], [v], 1.0, window=1)
    assert np.allclose(out[:, 0], [[3, 0], [8, 6]])
    out, _ = K.attention(q, [0, 2], [k[:, :1]], [v[:, :1]], 1.0)      # the first query stands before the first token
    assert np.allclose(out[:, 0], [[0, 0], [1, 0]])


def test_block_tables_hand_values():
    t = np.array([[7, -1, -1], [-1, -1, -1]])
    table, qs, kl, slots, pos, left = K.block_tables(np.array([15, 0]), np.array([2, 1]), np.array([4, 5, 6]), 3, 16, t, 4)
    assert table.tolist() == [[7, 6, -1], [5, -1, -1]] and left == 1
    assert qs.tolist() == [0, 2, 3] and kl.tolist() == [17, 1]
    assert slots.tolist() == [7 * 16 + 15, 6 * 16, 5 * 16, -1] and pos.tolist() == [15, 16, 0, 0]
