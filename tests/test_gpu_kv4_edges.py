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

from test_gpu_kv4 import U16, UBF, attend, bits, check, ints, make_batch, ok  # noqa: E402


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


# ------------------------------------------------------------------ one token has all of the weight
def cache_of(r, rows, P):
    """Pages and table that hold the given rows (float [2, hkv, n, D] for each request), and what they are after 4 bits:
    (pages, table, keys, values), float64, and the value rows' range 15 s."""
    hkv, D = rows[0].shape[1], rows[0].shape[3]
    blocks = [-(-x.shape[2] // P) for x in rows]
    pages = np.full((sum(blocks), hkv, P * (D + 8)), 0xFF, np.uint8)      # NaN pairs where there is no token
    perm, at = r.permutation(len(pages)), 0
    table = np.full((len(rows), max(blocks)), -1, np.int64)
    ks, vs, ranges = [], [], []
    for b, x in enumerate(rows):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
        u, s, z = K.quantise(x)
        words = (u.reshape(*u.shape[:3], -1, 8).astype(np.uint32) << K.BITS).sum(-1, dtype=np.uint32)
        for i in range(x.shape[2]):
            pg = pages[table[b, i // P]]
            for h in range(hkv):
                for side in range(2):
                    row = side * P + i % P
                    pg[h, row * D // 2:(row + 1) * D // 2] = words[side, h, i].view(np.uint8)
                    pg[h, P * D + 4 * row:P * D + 4 * row + 4] = np.stack([s[side, h, i], z[side, h, i]]).view(np.uint8)
        d = K.dequantise(u, s, z)
        ks.append(d[0])
        vs.append(d[1])
        ranges.append(15 * s[1].astype(np.float64))
    return pages.reshape(len(pages), -1), table, ks, vs, ranges


def one_hot_batch(r, kv, ql, hq, hkv, D, qscale, kscale):
    """Keys of random signs, and queries that have the signs of one token that they see each (their target); the token
    behind a query, hidden from it, has its first head's target's signs twice as large.  (rows of ones for the values,
    queries float, targets)"""
    g, rows, qs, targets = hq // hkv, [], [], []
    for n, m in zip(kv, ql):
        k = np.where(r.rand(hkv, n, D) < 0.5, -1.0, 1.0)
        q, t = np.zeros((m, hq, D)), np.zeros((m, hq), int)
        before = [r.permutation(n - m + 1) for _ in range(hkv)]   # the tokens before the call's, and its first one
        for i in range(m):
            for h in range(hq):                                   # (the first heads' own ones are shadowed, so no one else's)
                t[i, h] = before[h // g][i if h % g == 0 else r.randint(m, n - m + 1)]
                q[i, h] = k[h // g, t[i, h]] * r.uniform(0.75, 1.25, D)
        for i in range(m - 1):
            for h in range(hkv):
                k[h, n - m + i + 1] = 2 * k[h, t[i, h * g]]
        rows.append(np.stack([k * kscale, np.ones_like(k)]))
        qs.append(q * qscale)
        targets.append(t)
    return rows, np.concatenate(qs), targets


def lead_of(q, q_start, ks, targets, scale, causal=True):
    """How far the targets' scores are above all others that the query sees, in log2 units, at least; and what the queries
    should give: one target each."""
    least = np.inf
    for b, k in enumerate(ks):
        n, g = q_start[b + 1] - q_start[b], q.shape[1] // k.shape[0]
        for i in range(n):
            last = k.shape[1] - n + i + 1
            for h in range(q.shape[1]):
                s = k[h // g, :last] @ q[q_start[b] + i, h] * scale * np.log2(np.e)
                t = targets[b][i, h]
                least = min(least, s[t] - np.delete(s, t).max())
    return least


def one_hot_reference(q_shape, q_start, vs, ranges, targets):
    """The targets' value rows, and each row's range and largest magnitude [..., 2]."""
    ref, size = np.zeros(q_shape), np.zeros(q_shape[:2] + (2,))
    for b, v in enumerate(vs):
        g = q_shape[1] // v.shape[0]
        for i in range(q_start[b + 1] - q_start[b]):
            for h in range(q_shape[1]):
                t = targets[b][i, h]
                ref[q_start[b] + i, h] = v[h // g, t]
                size[q_start[b] + i, h] = ranges[b][h // g, t], np.abs(v[h // g, t]).max()
    return ref, size


def check_one_hot(out, ref, size, near=0.01):
    """One rounding to bf16; the value product's operands rounded to fp16 once each, the weight (times the row's scale, or
    alone) and the value: U16 of the row's range and twice U16 of the value; fp32 2^-20 of the row.  No error of the score
    is allowed: the other weights are nothing.  Zeros and the opposite signs are no answers within that, but for a share
    `near` of elements next to zero."""
    tol = UBF * np.abs(ref) * 1.01 + U16 * size[..., :1] + 2.02 * U16 * np.abs(ref) + 2.0 ** -20 * size[..., 1:]
    assert np.isfinite(out).all()
    assert (np.abs(out - ref) <= tol).all(), float((np.abs(out - ref) / tol).max())
    for wrong in (0 * ref, -ref):
        assert (np.abs(wrong - ref) <= tol).mean() < near


SATURATED = [(40.0, 1.0), (1e30, 1e-3), (1.5, 1000.0), (1.5, 20000.0), (300.0, 20.0)]


@pytest.mark.parametrize("kv,ql,hq,hkv,D,P", [
    ([150, 90], [1, 1], 4, 2, 128, 16), ([700], [5], 4, 1, 64, 32), ([150, 210], [60, 70], 4, 2, 128, 16), ([300], [130], 3, 1, 64, 64)])
@pytest.mark.parametrize("qscale,kscale", SATURATED)
def test_attention_saturated_scores(kv, ql, hq, hkv, D, P, qscale, kscale):
    """Where one token leads by far more than scores are off by, the answer is its value row, however large the scores."""
    r = np.random.RandomState(D + len(ql))
    rows, q, targets = one_hot_batch(r, kv, ql, hq, hkv, D, qscale, kscale)
    for x in rows:
        x[1] = r.randn(*x[1].shape) * np.exp(r.randn(*x[1].shape[:2], 1))
    pages, table, ks, vs, ranges = cache_of(r, rows, P)
    qb, qs = bits(q), np.concatenate([[0], np.cumsum(ql)]).astype(int)
    # scores are off by fp32's 2^-22 and, with keys in fp16, 2^-11 of their size, which is below the sum of 128 |q k|
    size = 2 * 1.25 * qscale * kscale * D * D ** -0.5 * np.log2(np.e)
    assert lead_of(synth.bf16_to_f64(qb), qs, ks, targets, D ** -0.5) > 40 + 2.0 ** -9 * size
    out = attend(pages, table, qb, qs, kv, hq, hkv, D, P, D ** -0.5)
    ok()
    check_one_hot(out, *one_hot_reference(out.shape, qs, vs, ranges, targets))


@pytest.mark.parametrize("kv,ql,hq,hkv,D,P,window", [
    ([400], [1], 1, 1, 64, 16, 0), ([400], [1], 4, 1, 128, 32, 390), ([150, 210], [4, 5], 4, 2, 128, 16, 0),
    ([900], [8], 4, 1, 64, 64, 0), ([150, 210], [60, 70], 4, 2, 128, 16, 0), ([400], [70], 2, 1, 64, 16, 0)])
@pytest.mark.parametrize("small", [2.0 ** -10, 2.0 ** -16])
def test_attention_small_values_of_the_token_that_counts(kv, ql, hq, hkv, D, P, window, small):
    """The targets' value rows are 2^10 or 2^16 times smaller than the other tokens', which have no weight, and the request's
    last and first tokens, hidden from the earlier queries or behind the window, are 256 times larger still: the answer keeps
    the precision of the targets' own rows."""
    r = np.random.RandomState(D + len(ql) + window)
    rows, q, targets = one_hot_batch(r, kv, ql, hq, hkv, D, 40.0, 2.0)
    for x, t in zip(rows, targets):
        x[1] = r.randn(*x[1].shape)
        x[1][:, [0, 1, -1]] *= 256
        for i, h in np.ndindex(*t.shape):
            if t[i, h] > 10:
                x[1][h // (hq // hkv), t[i, h]] = small * r.randn(D)
    pages, table, ks, vs, ranges = cache_of(r, rows, P)
    qb, qs = bits(q), np.concatenate([[0], np.cumsum(ql)]).astype(int)
    assert lead_of(synth.bf16_to_f64(qb), qs, ks, targets, D ** -0.5) > 60
    out = attend(pages, table, qb, qs, kv, hq, hkv, D, P, D ** -0.5, True, window)
    ok()
    keep = np.concatenate([(t > 10).reshape(-1) for t in targets]).reshape(out.shape[:2])
    ref, size = one_hot_reference(out.shape, qs, vs, ranges, targets)
    assert keep.mean() > 0.8
    check_one_hot(out[keep], ref[keep], size[keep])


@pytest.mark.parametrize("kv,ql,hq,hkv,D,P,window", [
    ([400], [1], 4, 1, 128, 32, 390), ([150, 210], [4, 5], 4, 2, 128, 16, 0), ([900], [8], 4, 1, 64, 64, 0),
    ([700], [3], 8, 1, 128, 16, 500), ([150, 210], [60, 70], 4, 2, 128, 16, 0)])
def test_attention_infinite_values_where_there_is_no_weight(kv, ql, hq, hkv, D, P, window):
    """Values of 1e38 (stored as 32768) in rows that a query does not see, or sees with no weight, leave it the precision of
    the rows that count, here a thousand times smaller than usual ones."""
    r = np.random.RandomState(D + len(ql) + window)
    rows, q, targets = one_hot_batch(r, kv, ql, hq, hkv, D, 40.0, 2.0)
    for x, t in zip(rows, targets):
        x[1] = 2.0 ** -10 * r.randn(*x[1].shape)
        free = np.setdiff1d(np.arange(x.shape[2]), t)
        x[1][:, free[::7], ::5] = 1e38                  # in every warp's and every block's share of the tokens
        x[1][:, free[3::7], ::3] = -1e38
    pages, table, ks, vs, ranges = cache_of(r, rows, P)
    qb, qs = bits(q), np.concatenate([[0], np.cumsum(ql)]).astype(int)
    assert lead_of(synth.bf16_to_f64(qb), qs, ks, targets, D ** -0.5) > 60
    out = attend(pages, table, qb, qs, kv, hq, hkv, D, P, D ** -0.5, True, window)
    ok()
    ref, size = one_hot_reference(out.shape, qs, vs, ranges, targets)
    seen = np.array([[not window or t[i, h] > n - m + i - window for h in range(hq)]
                     for n, m, t in zip(kv, ql, targets) for i in range(m)])
    assert seen.mean() > 0.5
    check_one_hot(out[seen], ref[seen], size[seen], near=0.05)      # few rows, of 16 levels each


@pytest.mark.parametrize("ql", [[1], [5], [80]])
@pytest.mark.parametrize("qscale,kscale", SATURATED + [(1e4, 5000.0), (1e5, 20000.0), (1e-3, 1e-3)])
def test_attention_equal_scores_of_any_size(ql, qscale, kscale):
    """All keys alike: every token that a query sees counts the same, whatever the scores' size and sign, and the values' sizes
    from 2^-20 to the largest that the cache holds."""
    kv, hq, hkv, D, P = [333], 4, 1, 64, 16
    r = np.random.RandomState(41)
    v = r.randn(333, D) * 2.0 ** r.randint(-20, 12, (333, 1))
    v[50], v[200, ::2], v[200, 1::2] = 1e38, 1e38, -1e38
    x = np.stack([np.broadcast_to(r.randn(D) * kscale, (1, 333, D)), v[None]])
    pages, table, ks, vs, ranges = cache_of(r, [x], P)
    q, qs = bits(r.randn(ql[0], hq, D) * qscale), [0, ql[0]]
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5)
    ok()
    for i in range(ql[0]):
        n = 333 - ql[0] + i + 1
        v, size = vs[0][0, :n], ranges[0][0, :n]
        ref = v.mean(0)
        # as check_one_hot, on the average; fp32's sums of values that cancel, 2^-20 of the largest
        tol = UBF * np.abs(ref) * 1.01 + U16 * size.mean() + 2.02 * U16 * np.abs(v).mean(0) + 2.0 ** -20 * np.abs(v).max()
        assert np.isfinite(out[i]).all() and (np.abs(out[i] - ref) <= tol).all(), float((np.abs(out[i] - ref) / tol).max())


@pytest.mark.parametrize("ql", [[1], [5], [80]])
def test_attention_reads_scales_of_either_sign(ql):
    """The writer stores scales of 0 and above; a cache filled elsewhere may hold value rows upside down, s u + z with s < 0."""
    kv, hq, hkv, D, P = [200], 4, 1, 64, 16
    r = np.random.RandomState(43)
    pages, table, ks, vs, ranges = cache_of(r, [np.stack([r.randn(1, 200, D), r.randn(1, 200, D) * np.exp2(r.randint(-4, 12, (1, 200, 1)))])], P)
    heads = pages.reshape(len(pages), P * (D + 8))
    for b, i in np.ndindex(len(pages), P):
        sz = heads[b, P * D + 4 * (P + i):][:4].view(np.float16)
        if np.isfinite(sz).all() and i % 3:
            sz[:] = -sz[0], -sz[1]                                  # every third row as it was
    q, qs = bits(r.randn(ql[0], hq, D)), [0, ql[0]]
    k, v = K.unpack(pages, table[0], 200, P, hkv, D)
    assert (v == np.where(np.arange(200)[:, None] % P % 3, -vs[0][0], vs[0][0])).all()
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, [k], [v], D ** -0.5)
    check(out, ref, spread)


# ------------------------------------------------------------------ pages of several requests, calls in flight together
@pytest.mark.parametrize("ql", [[1, 1, 1], [3, 1, 70], [60, 70, 50]])
def test_requests_that_share_pages(ql):
    """A common prefix is held once: the tables of several requests name the same pages."""
    common, own, hq, hkv, D, P = 160, [41, 70, 77], 4, 2, 128, 16
    r = np.random.RandomState(51)
    pages, table, ks, vs, _ = cache_of(r, [r.randn(2, hkv, n, D) for n in [common] + own], P)
    rows = np.full((3, common // P + table.shape[1]), -1)
    for b in range(3):
        n = -(-own[b] // P)
        rows[b, :common // P], rows[b, common // P:common // P + n] = table[0, :common // P], table[b + 1, :n]
    kv = [common + n for n in own]
    q, qs = bits(r.randn(sum(ql), hq, D)), np.concatenate([[0], np.cumsum(ql)]).astype(int)
    out = attend(pages, rows, q, qs, kv, hq, hkv, D, P, D ** -0.5)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, *([np.concatenate([x[0], x[b + 1]], 1) for b in range(3)] for x in (ks, vs)),
                              D ** -0.5)
    check(out, ref, spread)


def test_two_streams_at_once():
    """Calls in flight on two streams, each with its own workspace, give the bits that they give alone."""
    hq, hkv, D, P = 8, 2, 128, 16
    calls = []
    for seed, kv, ql in ((61, [900, 70, 2000, 1] * 8, [1, 1, 3, 1] * 8), (62, [300, 500, 40] * 4, [200, 1, 40] * 4)):
        r = np.random.RandomState(seed)
        pages, table, _, _, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
        cache, mq, mk = Q.Kv4Cache(torch.from_numpy(pages).cuda(), P, hkv, D), max(ql), max(kv)
        qt = bf16_tensor(q).view(torch.bfloat16).view(-1, hq, D)
        ws = torch.empty(Q.kv4_attention_ws_size(len(kv), hq, hkv, D, qt.shape[0], mq, mk), dtype=torch.uint8, device="cuda")
        args = (cache, qt, ints(qs), ints(kv), ints(table))
        calls.append((torch.cuda.Stream(), lambda out, args=args, ws=ws, mq=mq, mk=mk: Q.kv4_attention(*args, out, ws, mq, mk, D ** -0.5), qt))
    alone = [call(torch.empty_like(qt)) for _, call, qt in calls]
    outs = [[torch.full_like(qt, float("nan")) for _ in range(20)] for _, _, qt in calls]
    torch.cuda.synchronize()
    for i in range(20):
        for (stream, call, _), out in zip(calls, outs):
            with torch.cuda.stream(stream):
                call(out[i])
    torch.cuda.synchronize()
    ok()
    for first, out in zip(alone, outs):
        assert bool(first.isfinite().all()) and all(torch.equal(first, o) for o in out)


def test_errors_of_two_kinds_are_each_cleared():
    """The status call gives one error, clears all words that hold one, and then says that all is well."""
    cache = Q.Kv4Cache.empty(2, 16, 1, 64)
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        Q.kv4_append(cache, k, k, ints([99]))                                                       # EINVAL, cache kernels
        ws = torch.empty(Q.kv4_attention_ws_size(1, 1, 1, 64, 1, 1, 5), dtype=torch.uint8, device="cuda")
        Q.kv4_attention(cache, k, ints([0, 1]), ints([9]), ints([[0]]), k.clone(), ws, 1, 5, 1.0)   # ECAPACITY, attention
        assert Q.qmoe_check_status() == Q.QMOE_EINVAL
        ok()


@pytest.mark.parametrize("ql", [[12, 2], [90, 5]])
def test_widest_window_with_queries_before_the_first_token(ql):
    """A window one below the largest bound, and queries that stand before the first token: these see nothing, the others all."""
    kv, hq, hkv, D, P = [4, 70], 4, 2, 64, 16
    r = np.random.RandomState(71)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, 0.125, window=2 ** 31 - 2, max_kv=2 ** 31 - 1)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, 0.125)
    check(out, ref, spread)
    assert not out[:ql[0] - 4].any()


@pytest.mark.parametrize("kv,ql,P,window,gone", [
    ([700, 90], [1, 1], 16, 300, -1), ([700, 390], [3, 2], 16, 300, 10 ** 6), ([500], [1], 32, 100, -1), ([900, 300], [70, 80], 16, 200, -1),
    ([900], [100], 64, 130, -1)])
@pytest.mark.parametrize("causal", [True, False])
def test_pages_behind_the_window_may_be_gone(kv, ql, P, window, gone, causal):
    """Blocks that no query of the request sees any more need no page: neither an error nor a change."""
    hq, hkv, D = 4, 2, 128
    r = np.random.RandomState(81)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    dropped = 0
    for b, (n, m) in enumerate(zip(kv, ql)):
        first = K.visible(n, m, 0, causal, window)[0]
        table[b, :first // P] = gone
        dropped += first // P
    assert dropped
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, causal, window)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5, causal, window)
    check(out, ref, spread)
    table[0, kv[0] // P - 1] = -1                       # one that is seen is still missed
    attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, causal, window)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
