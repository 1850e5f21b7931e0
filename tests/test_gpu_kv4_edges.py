"""GPU parity of attention over the 4-bit cache where it can go wrong beside the shapes of test_gpu_kv4: long runs of short
items, values of very different sizes, saturated scores, host-side bounds, shared pages, streams."""
import numpy as np
import pytest

import synth
from oracle import kv4 as K

from helpers import bf16_tensor

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
Q = pytest.importorskip("decode_matvec_gb300")

from test_gpu_kv4 import attend, bits, check, ints, make_batch, ok  # noqa: E402


@pytest.mark.parametrize("B,q_hi,kv_hi,hq,hkv,D,P,window", [
    (70, 70, 200, 32, 8, 128, 16, 0),       # several items a block, one or two tiles of keys each
    (70, 70, 200, 32, 8, 128, 32, 40),      # the same behind a window, single tokens among them
    (230, 9, 300, 34, 1, 64, 64, 0),        # groups that only the tiles take
])
def test_tiles_many_short_items(B, q_hi, kv_hi, hq, hkv, D, P, window):
    """A block goes through several items of the tile path one after another, and takes up each where the last one ended."""
    r = np.random.RandomState(B + D + window)
    ql = r.randint(1, q_hi + 1, B)
    ql[::5] = 1
    kv = (ql + r.randint(0, kv_hi - q_hi, B)).tolist()
    ql = ql.tolist()
    assert sum(-(-n * (hq // hkv) // 256) for n in ql if n * (hq // hkv) > 32 or hq // hkv > 32) * hkv > 152
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, True, window)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5, True, window)
    check(out, ref, spread)


@pytest.mark.parametrize("window", [0, 2 ** 31 - 200])
def test_bounds_at_the_end_of_int32_choose_as_any_large_bound_does(window):
    """max_kv is a bound, not a length: one that says "no bound" gives the same blocks, hence the same bits, as one that is large."""
    kv, ql, hq, hkv, D, P = [5000, 3000], [1, 1], 4, 2, 128, 64
    r = np.random.RandomState(31)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    large = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, max_kv=2 ** 31 - 128)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, window=window, max_kv=2 ** 31 - 1)
    ok()
    assert np.array_equal(out, large)
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5)
    check(out, ref, spread)


@pytest.mark.parametrize("ql", [[1, 1], [1, 40]])
def test_lengths_past_the_last_whole_tile_of_int32_are_reported(ql):
    """2^31 - 1 tokens, which no table here can hold, are an error and not one tile of them."""
    kv, hq, hkv, D, P = [50, 60], 2, 1, 64, 16
    r = np.random.RandomState(32)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    out = attend(pages, table, q, qs, [50, 2 ** 31 - 1], hq, hkv, D, P, 0.125, max_kv=2 ** 31 - 1, fill=7.0)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    ref, spread = K.attention(synth.bf16_to_f64(q[:1]), [0, 1], ks[:1], vs[:1], 0.125)
    check(out[:1], ref, spread)
    assert (out[1:] == 7).all()


@pytest.mark.parametrize("tokens", [20, 5000])
def test_block_tables_do_not_read_past_the_stack(tokens):
    """A count of free pages above the stack's places: an error, and the pages are those that the stack has."""
    P, n = 16, -(-tokens // 16)
    stack = np.arange(100, 100 + n + 3)
    memory = ints(np.concatenate([stack, np.full(50, 7)]))         # what lies behind the stack is not a page of it
    cached, new, nf, out = ints([0]), ints([tokens]), ints([len(stack) + 40]), ints([0])
    table, qs, kl = ints(np.full((1, n), -1)), ints([0, 0]), ints([0])
    sl, po = ints(np.zeros(tokens)), ints(np.zeros(tokens))
    Q.kv4_block_tables(cached, new, memory[:len(stack)], nf, P, table, qs, kl, sl, po, out)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    assert table.cpu().numpy()[0].tolist() == stack[::-1][:n].tolist() and out.item() == len(stack) - n
    assert np.array_equal(sl.cpu().numpy(), table.cpu().numpy()[0][np.arange(tokens) // P] * P + np.arange(tokens) % P)
    nf.fill_(len(stack))
    Q.kv4_block_tables(cached, new, memory[:len(stack)], nf, P, table, qs, kl, sl, po, out)
    ok()
