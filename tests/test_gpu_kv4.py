"""GPU parity of the 4-bit paged cache operators with the float64 oracle, and their refusals."""
import numpy as np
import pytest

import synth
from oracle import kv4 as K

from helpers import bf16_tensor, bf16_values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
Q = pytest.importorskip("decode_matvec_gb300")

U16 = 2.0 ** -11      # unit roundoff of fp16
UBF = 2.0 ** -8       # of bf16 (8 significant bits)


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def bits(x):
    """bf16 bits of float values that need not be exact."""
    return (K.bf16_round(x).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def ok():
    assert Q.qmoe_check_status() == Q.QMOE_OK, Q.qmoe_last_error()


# ------------------------------------------------------------------ block tables
def run_tables(cached, new, free, n_free, P, table, n_tokens, alias=False):
    cached, new = np.asarray(cached), np.asarray(new)
    B = len(cached)
    t = ints(table)
    nf = ints([n_free])
    out = nf if alias else ints([-5])
    qs, kl = ints(np.full(B + 1, -9)), ints(np.full(B, -9))
    sl, po = ints(np.full(n_tokens, -9)), ints(np.full(n_tokens, -9))
    Q.kv4_block_tables(ints(cached), ints(new), ints(free), nf, P, t, qs, kl, sl, po, out)
    return [x.cpu().numpy() for x in (t, qs, kl, sl, po)] + [int(out.item())]


@pytest.mark.parametrize("B,lo,hi,chi,P,pad,alias", [
    (1, 1, 1, 0, 16, 0, False), (1, 0, 0, 40, 16, 3, True), (8, 1, 1, 200, 16, 0, True), (33, 0, 70, 100, 32, 5, False),
    (1024, 0, 3, 300, 64, 0, True), (1025, 0, 9, 50, 16, 1, False), (3000, 1, 1, 70, 32, 0, True),
    (5, 500, 4000, 17, 64, 0, False), (40, 16, 16, 0, 16, 7, False)])
def test_block_tables(B, lo, hi, chi, P, pad, alias):
    r = np.random.RandomState(B + P)
    cached, new = r.randint(0, chi + 1, B), r.randint(lo, hi + 1, B)
    have, want = -(-cached // P), -(-(cached + new) // P)
    perm = r.permutation(int(want.sum()) + 4)
    table = np.full((B, int(want.max()) + 2), -7, np.int64)
    at = 0
    for b in range(B):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    free = perm[at:]
    n = int(new.sum()) + pad
    got = run_tables(cached, new, free, len(free), P, table, n, alias)
    ref = K.block_tables(cached, new, free, len(free), P, table, n)
    for g, e in zip(got, ref):
        assert np.array_equal(g, e)
    ok()


def test_block_tables_out_of_pages_and_out_of_room():
    table = np.full((3, 4), -1)
    got = run_tables([0, 0, 0], [20, 20, 20], [3, 4, 5], 3, 16, table, 60)
    ref = K.block_tables(np.zeros(3, int), np.full(3, 20), np.array([3, 4, 5]), 3, 16, table, 60)
    for g, e in zip(got, ref):
        assert np.array_equal(g, e)
    assert Q.qmoe_check_status() == Q.QMOE_ECAPACITY
    got = run_tables([0], [20], [3, 4, 5], 3, 16, table[:1], 7)        # more tokens than the arrays hold
    assert got[3].tolist() == [5 * 16 + i for i in range(7)] and got[1].tolist() == [0, 7]
    assert Q.qmoe_check_status() == Q.QMOE_ECAPACITY
    got = run_tables([-3, 2], [4, -1], [3, 4, 5], 3, 16, np.full((2, 1), 9), 4)   # negative lengths are read as 0
    assert got[2].tolist() == [4, 2] and got[3].tolist() == [5 * 16 + i for i in range(4)]
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    got = run_tables([0], [40], [3, 4, 5], 3, 16, np.full((1, 2), -1), 40)        # three blocks, a table of two
    assert (got[3][:32] >= 0).all() and (got[3][32:] == -1).all()
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL


# ------------------------------------------------------------------ norm and rotation
def cos_sin(n_pos, rot):
    ang = np.arange(n_pos)[:, None] * (10000.0 ** (-np.arange(0, rot, 2) / rot))[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.parametrize("T,hq,hkv,D,rot,inter,norm,extra", [
    (1, 16, 16, 128, 128, False, True, 0), (1, 1, 1, 64, 64, True, True, 0), (7, 5, 1, 128, 64, False, True, 8),
    (33, 6, 3, 64, 32, True, False, 64), (3, 4, 2, 128, 0, False, True, 0), (130, 2, 2, 64, 16, False, True, 0),
    (19, 8, 8, 128, 48, False, True, 0), (65, 3, 1, 64, 48, True, True, 24)])
def test_qk_norm_rope(T, hq, hkv, D, rot, inter, norm, extra):
    r = np.random.RandomState(T * 100 + D)
    width = (hq + 2 * hkv) * D + extra
    x = bits(r.randn(T, width) * np.exp(r.randn(T, 1)))
    wq, wk = bits(1 + 0.3 * r.randn(D)), bits(1 + 0.3 * r.randn(D))
    cs = cos_sin(500, rot) if rot else None
    pos = r.randint(0, 500, T)
    q, k = (torch.full((T, h, D), float("nan"), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    Q.qk_norm_rope(bf16_tensor(x), hq, hkv, D, bf16_tensor(wq) if norm else None, bf16_tensor(wk) if norm else None, 1e-5,
                   None if cs is None else torch.from_numpy(cs).cuda(), ints(pos), q, k, interleaved=inter)
    ok()
    xf = synth.bf16_to_f64(x)[:, :(hq + hkv) * D].reshape(T, hq + hkv, D)
    for got, part, w in ((q, xf[:, :hq], wq), (k, xf[:, hq:], wk)):
        ref = K.norm_rope(part, synth.bf16_to_f64(w) if norm else None, 1e-5, None if cs is None else cs.astype(np.float64), pos, inter)
        # one rounding to bf16 plus fp32 arithmetic: a rotation's two products may cancel, so the fp32 part scales with the pair
        big = np.abs(ref).max(-1, keepdims=True) * 2
        assert (np.abs(got.double().cpu().numpy() - ref) <= UBF * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -20 * big).all()


def test_qk_norm_rope_writes_the_cache_as_append_does():
    r = np.random.RandomState(3)
    T, hq, hkv, D, P = 37, 8, 2, 128, 16
    x = bf16_tensor(bits(r.randn(T, (hq + 2 * hkv) * D)))
    w = bf16_tensor(bits(1 + 0.3 * r.randn(D)))
    cs, pos = torch.from_numpy(cos_sin(64, D)).cuda(), ints(r.randint(0, 64, T))
    slots = ints(np.where(np.arange(T) % 9 == 4, -1, r.permutation(4 * P)[:T]))
    a, b = Q.Kv4Cache.empty(4, P, hkv, D), Q.Kv4Cache.empty(4, P, hkv, D)
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((T, hkv, D), dtype=torch.bfloat16, device="cuda")
    Q.qk_norm_rope(x, hq, hkv, D, w, w, 1e-5, cs, pos, q, k, cache=a, slots=slots)
    Q.kv4_append(b, k, x.view(torch.bfloat16)[:, (hq + hkv) * D:].reshape(T, hkv, D), slots)
    q2 = torch.empty_like(q)
    Q.qk_norm_rope(x, hq, hkv, D, w, w, 1e-5, cs, pos, q2, None, cache=a, slots=slots)    # k_out left out
    ok()
    assert torch.equal(a.pages, b.pages) and bool(a.pages.any()) and torch.equal(q, q2)


def test_qk_norm_rope_position_outside_the_table():
    x = bf16_tensor(bits(np.ones((2, 3 * 64))))
    q, k = (torch.empty((2, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q.qk_norm_rope(x, 1, 1, 64, None, None, 0.0, torch.from_numpy(cos_sin(10, 64)).cuda(), ints([10, -1]), q, k)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    ref = K.norm_rope(np.ones((2, 1, 64)), None, 0, cos_sin(10, 64).astype(float), np.array([9, 0]), False)
    assert np.abs(q.double().cpu().numpy() - ref).max() <= UBF


# ------------------------------------------------------------------ cache write and read
@pytest.mark.parametrize("T,hkv,D,P", [(1, 1, 64, 16), (1, 16, 128, 64), (64, 3, 64, 32), (129, 4, 128, 16), (50, 5, 64, 64)])
def test_append_is_bit_exact_and_gather_reads_it_back(T, hkv, D, P):
    r = np.random.RandomState(T + D + P)
    x = r.randn(T, 2, hkv, D) * np.exp(2 * r.randn(T, 2, hkv, 1))
    x[r.rand(*x.shape) < 0.01] *= 30
    x[0, 0, 0] = 3.25                                         # a constant row
    if T > 3:
        x[1, 1, 0, :4] = [np.nan, np.inf, -np.inf, 1e38]
        x[2, 0, 0] = 1e-6 * r.randn(D)                        # below fp16's normal range
        x[3, 0, 0] = 0
    xb = bits(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf))
    xb[np.isnan(x)] = 0x7FC1
    n_pages = -(-T // P) + 2
    slots = r.permutation(n_pages * P)[:T]
    skip = np.arange(T) % 11 == 5
    slots[skip] = -1
    cache = Q.Kv4Cache(torch.full((n_pages, Q.Kv4Cache.page_bytes(P, hkv, D)), 0xAB, dtype=torch.uint8, device="cuda"), P, hkv, D)
    kv = bf16_tensor(xb.reshape(T, -1)).view(T, 2, hkv, D)
    Q.kv4_append(cache, kv[:, 0], kv[:, 1], ints(slots))
    ok()
    xf = synth.bf16_to_f64(xb)
    u, s, z = K.quantise(xf)
    got = cache.pages.cpu().numpy().reshape(n_pages, hkv, -1)
    ref = np.full_like(got, 0xAB)
    for t in range(T):                                        # place the rows one by one
        if skip[t]:
            continue
        pg, i = divmod(int(slots[t]), P)
        for h in range(hkv):
            for side in range(2):
                one = K.pack_page(*[np.repeat(a[t, side, h][None], 16, 0) for a in (u, s, z)] * 2)
                w = one[:D // 2]
                ref[pg, h, (side * P + i) * (D // 2):][:D // 2] = w
                pair = np.stack([s[t, side, h], z[t, side, h]]).view(np.uint8)
                ref[pg, h, P * D + 4 * (side * P + i):][:4] = pair
    assert np.array_equal(got, ref)
    k, v = (torch.full((T, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q.kv4_gather(cache, ints(slots), k, v)
    ok()
    val = K.bf16_round(K.dequantise(u, s, z))
    val[skip] = 0
    assert np.array_equal(k.double().cpu().numpy(), val[:, 0]) and np.array_equal(v.double().cpu().numpy(), val[:, 1])


def test_append_and_gather_refuse_slots_outside_the_cache():
    cache = Q.Kv4Cache.empty(2, 16, 1, 64)
    k = bf16_tensor(bits(np.ones((3, 64)))).view(3, 1, 64)
    Q.kv4_append(cache, k, k, ints([32, -2, 31]))
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    out = torch.full((3, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    o2 = out.clone()
    Q.kv4_gather(cache, ints([31, 32, 2 ** 31 - 1]), out, o2)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    assert bool((out[0] == 1).all()) and not bool(out[1:].any()) and not bool(o2[1:].any())
    Q.kv4_append(cache, k[:0], k[:0], ints([]))
    ok()


# ------------------------------------------------------------------ attention
def make_batch(r, kv, ql, hq, hkv, D, P, qscale=1.5, kscale=1.0, vscale=1.0, garbage=True):
    """A cache of random rows in shuffled pages (unused places full of NaN pairs), and the batch that reads it."""
    blocks = [-(-n // P) for n in kv]
    n_pages = sum(blocks) + 2
    pages = r.randint(0, 256, (n_pages, hkv, P * (D + 8))).astype(np.uint8)
    perm = r.permutation(n_pages)
    table = np.full((len(kv), max(blocks + [1]) + 1), -1, np.int64)
    at, ks, vs = 0, [], []
    pages[:, :, P * D:] = np.full(1, np.nan if garbage else 0, np.float16).view(np.uint8).tolist() * (4 * P)
    for b, n in enumerate(kv):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
        x = r.randn(2, hkv, n, D)
        x[0] *= kscale
        x[1] *= vscale
        x[:, :, :, 3] *= 4
        u, s, z = K.quantise(x)
        for i in range(n):
            pg = pages[table[b, i // P]]
            for h in range(hkv):
                for side in range(2):
                    w = (u[side, h, i].reshape(-1, 8).astype(np.uint32) << K.BITS).sum(-1, dtype=np.uint32)
                    row = side * P + i % P
                    pg[h, row * D // 2:(row + 1) * D // 2] = w.view(np.uint8)
                    pg[h, P * D + 4 * row:P * D + 4 * row + 4] = np.stack([s[side, h, i], z[side, h, i]]).view(np.uint8)
        d = K.dequantise(u, s, z)
        ks.append(d[0])
        vs.append(d[1])
    q = bits(r.randn(sum(ql), hq, D) * qscale)
    return pages.reshape(n_pages, -1), table, ks, vs, q, np.concatenate([[0], np.cumsum(ql)]).astype(int)


def attend(pages, table, q, q_start, kv, hq, hkv, D, P, scale, causal=True, window=0, max_q=None, max_kv=None, fill=float("nan")):
    cache = Q.Kv4Cache(torch.from_numpy(pages).cuda(), P, hkv, D)
    qt = bf16_tensor(q).view(torch.bfloat16).view(-1, hq, D)
    out = torch.full_like(qt, fill)
    mq = int(np.diff(q_start).max()) if max_q is None else max_q
    mk = max(list(kv) + [0]) if max_kv is None else max_kv
    n = Q.kv4_attention_ws_size(len(kv), hq, hkv, D, qt.shape[0], mq, mk)
    ws = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device="cuda")      # NaNs
    Q.kv4_attention(cache, qt, ints(q_start), ints(kv), ints(table), out, ws, mq, mk, scale, causal=causal, window=window)
    assert bool((ws[n:] == 0xFF).all())
    return out.double().cpu().numpy()


def check(out, ref, spread, norm=True):
    """Element by element: one rounding to bf16, UBF |out|; as |out| <= max |v|, half of it is counted as UBF / 2 max |v| =
    4 U16 max |v|, which covers what follows for the probabilities and values too.  Keys, values and probabilities rounded to fp16 at most once each (a score
    moves by at most U16 * scale * sum |q k|, an output by twice that times max |v|); 2^-13 max |v| for fp32.  Over all: bf16's rms plus a margin for the rest."""
    tol = UBF / 2 * np.abs(ref) * 1.01 + (2.02 * U16 * spread[..., :1] + (4 * U16 + 2.0 ** -13) * spread[..., 1:]) + 1e-30
    assert np.isfinite(out).all()
    assert (np.abs(out - ref) <= tol).all(), float((np.abs(out - ref) / tol).max())
    if norm and ref.size >= 1024 and np.linalg.norm(ref) > 0:
        assert np.linalg.norm(out - ref) / np.linalg.norm(ref) <= 2.5e-3


CASES = [
    # kv lengths, query lengths, hq, hkv, D, page, causal, window
    ([1], [1], 1, 1, 64, 16, True, 0),
    ([1], [1], 16, 16, 128, 64, True, 0),
    ([17, 1, 64, 65, 300], [1] * 5, 8, 2, 128, 16, True, 0),
    ([0, 5, 0, 63], [1] * 4, 4, 4, 64, 32, True, 0),
    ([500, 33], [1, 1], 6, 2, 64, 64, True, 0),
    ([257], [1], 5, 1, 128, 16, True, 0),
    ([700, 129], [1, 1], 16, 1, 128, 32, True, 0),
    ([640], [1], 33, 1, 64, 16, True, 0),
    ([400], [1], 128, 1, 128, 16, True, 0),
    ([130, 40, 7], [3, 1, 5], 8, 4, 128, 16, True, 0),
    ([3, 2, 900], [5, 2, 4], 8, 1, 64, 64, True, 0),          # queries before the first token
    ([600, 90, 20], [1, 1, 1], 8, 2, 128, 16, True, 33),
    ([600, 90, 20], [4, 2, 1], 8, 2, 64, 32, True, 100),
    ([90, 20], [4, 9], 4, 2, 128, 16, False, 0),
    ([90, 20], [4, 9], 4, 2, 64, 16, False, 16),
    ([100], [100], 2, 1, 128, 64, True, 0),
    ([129, 257], [129, 200], 2, 2, 64, 16, True, 0),
    ([300, 40, 1], [150, 1, 1], 4, 1, 128, 32, True, 0),       # a prompt and two single tokens together
    ([513], [260], 3, 1, 128, 64, True, 0),
    ([400, 100], [140, 100], 4, 2, 64, 64, True, 50),
    ([200], [270], 2, 1, 128, 16, True, 0),                   # more queries than tokens
    ([333], [70], 7, 1, 128, 16, False, 0),
    ([260], [131], 2, 2, 128, 16, False, 77),
    ([50, 0, 60], [40, 0, 0], 4, 2, 128, 16, True, 0),        # requests without queries
    ([1100], [3], 40, 2, 128, 64, True, 0),
    ([2100, 5], [1, 1], 4, 4, 64, 16, True, 0),
]


@pytest.mark.parametrize("kv,ql,hq,hkv,D,P,causal,window", CASES)
def test_attention(kv, ql, hq, hkv, D, P, causal, window):
    r = np.random.RandomState(sum(kv) + hq + D)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, causal, window)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5, causal, window)
    check(out, ref, spread)
    empty = spread[..., 1] == 0
    assert not out[empty].any()


@pytest.mark.parametrize("ql", [[1, 1], [60, 70]])
@pytest.mark.parametrize("qscale,kscale,vscale", [(40.0, 1.0, 1.0), (1e30, 1e-3, 1.0), (1e-6, 1.0, 1.0), (1.5, 1000.0, 500.0),
                                                  (3e-4, 5000.0, 0.01)])
def test_attention_ranges(ql, qscale, kscale, vscale):
    kv, hq, hkv, D, P = [150, 90], 4, 2, 128, 16
    r = np.random.RandomState(5)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P, qscale, kscale, vscale)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5)
    # a score of magnitude S carries fp32's 2^-23 S of its own sums; past that nothing can be asked of a softmax
    spread[..., 0] = np.minimum(spread[..., 0] * (1 + 2.0 ** -11), spread[..., 1] / U16)
    check(out, ref, spread, norm=False)


@pytest.mark.parametrize("ql", [[1], [70]])
def test_attention_small_values_and_one_far_score(ql):
    """One token takes nearly all the weight and has values a thousand times smaller than the rest."""
    D, P, n = 64, 16, 400
    r = np.random.RandomState(6)
    pages, table, ks, vs, q, qs = make_batch(r, [n], ql, 1, 1, D, P, qscale=2.0)
    out = attend(pages, table, q, qs, [n], 1, 1, D, P, 1.0)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, 1.0)
    check(out, ref, spread, norm=False)


def test_attention_same_bits_again_and_on_another_stream():
    kv, ql, hq, hkv, D, P = [900, 70, 333, 1], [1, 1, 40, 1], 8, 2, 128, 16
    r = np.random.RandomState(9)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    first = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5)
    for _ in range(2):
        assert np.array_equal(first, attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5)
    assert np.array_equal(first, again)
    # larger bounds than the lengths need change nothing but the work
    wide = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, max_q=64, max_kv=3000)
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5)
    check(wide, ref, spread)


def test_attention_leaves_other_rows_and_reports_bad_tables():
    kv, ql, hq, hkv, D, P = [40, 60], [2, 3], 2, 1, 64, 16
    r = np.random.RandomState(10)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    extra = np.concatenate([q, q[:2]])
    out = attend(pages, table, extra, qs, kv, hq, hkv, D, P, 0.125, fill=7.0)
    assert (out[5:] == 7).all()
    ok()
    bad = table.copy()
    bad[1, 0] = len(pages)                     # a page outside the cache: its tokens are not seen
    out = attend(pages, bad, q, qs, kv, hq, hkv, D, P, 0.125)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, 0.125)
    check(out[:2], ref[:2], spread[:2])
    k1, v1 = ks[1][:, 16:], vs[1][:, 16:]
    ref, spread = K.attention(synth.bf16_to_f64(q[2:]), [0, 3], [k1], [v1], 0.125)
    check(out[2:], ref, spread)
    order = qs.copy()
    order[1] = 9                               # q_start out of order: those requests are skipped
    out = attend(pages, table, q, order, kv, hq, hkv, D, P, 0.125, max_q=3, fill=7.0)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL and (out == 7).all()


def test_attention_reports_lengths_past_its_bounds():
    kv, ql, hq, hkv, D, P = [200], [1], 2, 1, 64, 16
    r = np.random.RandomState(11)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    attend(pages, table, q, qs, kv, hq, hkv, D, P, 0.125, max_kv=100)
    assert Q.qmoe_check_status() == Q.QMOE_ECAPACITY
    attend(pages, table[:, :3], q, qs, kv, hq, hkv, D, P, 0.125)       # a table too short for the length
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL


def test_cache_past_32_bit_offsets():
    """Pages more than 2^32 bytes into the cache are written and read at their place."""
    P, hkv, D = 64, 16, 128
    n_pages = (5 << 30) // Q.Kv4Cache.page_bytes(P, hkv, D)
    cache = Q.Kv4Cache.empty(n_pages, P, hkv, D)
    r = np.random.RandomState(12)
    kv = r.randn(70, 2, hkv, D)
    kvt = bf16_tensor(bits(kv).reshape(70, -1)).view(70, 2, hkv, D)
    table = np.array([[n_pages - 1, n_pages - 3]])
    slots = table[0][np.arange(70) // P] * P + np.arange(70) % P
    Q.kv4_append(cache, kvt[:, 0], kvt[:, 1], ints(slots))
    u, s, z = K.quantise(K.bf16_round(kv))
    d = K.dequantise(u, s, z)
    for n in (1, 40):
        q = bits(r.randn(n, hkv, D))
        qt = bf16_tensor(q).view(torch.bfloat16).view(n, hkv, D)
        out = torch.empty_like(qt)
        ws = torch.empty(Q.kv4_attention_ws_size(1, hkv, hkv, D, n, n, 70) + 1, dtype=torch.uint8, device="cuda")
        Q.kv4_attention(cache, qt, ints([0, n]), ints([70]), ints(table), out, ws, n, 70, D ** -0.5)
        ok()
        ref, spread = K.attention(synth.bf16_to_f64(q), [0, n], [d[:, 0].transpose(1, 0, 2)], [d[:, 1].transpose(1, 0, 2)], D ** -0.5)
        check(out.double().cpu().numpy(), ref, spread)


# ------------------------------------------------------------------ refusals
def test_refusals():
    def refused(status, fn):
        with pytest.raises(Q.QmoeError) as e:
            fn()
        assert e.value.status == status
    cache = Q.Kv4Cache.empty(2, 16, 1, 64)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    good = (ints([0, 1]), ints([1]), ints([[0]]))
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_attention(cache, q, *good, q.clone(), ws, 1, 1, 1.0, window=-1))
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_attention(cache, q, *good, q.clone(), ws, -1, 1, 1.0))
    two = Q.Kv4Cache.empty(2, 16, 2, 64)
    q3 = torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda")
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_attention(two, q3, *good, q3.clone(), ws, 1, 1, 1.0))
    q129 = torch.zeros((1, 129, 64), dtype=torch.bfloat16, device="cuda")
    refused(Q.QMOE_EUNSUPPORTED, lambda: Q.kv4_attention(cache, q129, *good, q129.clone(), ws, 1, 1, 1.0))
    n = Q.kv4_attention_ws_size(1, 1, 1, 64, 1, 1, 100000)
    if n:
        refused(Q.QMOE_ECAPACITY, lambda: Q.kv4_attention(cache, q, *good, q.clone(), ws[:16], 1, 100000, 1.0))
    odd = torch.zeros(65 * 8, dtype=torch.bfloat16, device="cuda")[1:65].view(1, 1, 64)
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_attention(cache, odd, *good, q.clone(), ws, 1, 1, 1.0))
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_append(cache, odd, odd, ints([0])))
    bad = Q.Kv4Cache.empty(2, 24, 1, 64)
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_append(bad, q, q, ints([0])))
    d96 = Q.Kv4Cache.empty(2, 16, 1, 96)
    refused(Q.QMOE_EUNSUPPORTED, lambda: Q.kv4_append(d96, torch.zeros((1, 1, 96), dtype=torch.bfloat16, device="cuda"),
                                                      torch.zeros((1, 1, 96), dtype=torch.bfloat16, device="cuda"), ints([0])))
    x = torch.zeros((1, 192), dtype=torch.bfloat16, device="cuda")
    cs = torch.zeros((4, 24), device="cuda")
    refused(Q.QMOE_EINVAL, lambda: Q.qk_norm_rope(x, 1, 1, 64, None, None, 0.0, cs, ints([0]), q, q.clone()))
    refused(Q.QMOE_EINVAL, lambda: Q.qk_norm_rope(x, 1, 1, 64, None, None, 0.0, None, None, q, q.clone(), cache=cache))
    refused(Q.QMOE_EINVAL, lambda: Q.kv4_block_tables(ints([0]), ints([1]), ints([0]), ints([1]), 48, ints([[0]]), ints([0, 0]),
                                                      ints([0]), ints([0]), ints([0]), ints([0])))
    with pytest.raises(ValueError):
        Q.kv4_attention(cache, torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda"), *good, q.clone(), ws, 1, 1, 1.0)
    with pytest.raises(ValueError):
        Q.Kv4Cache(torch.zeros((2, 7), dtype=torch.uint8, device="cuda"), 16, 1, 64)
    ok()


# ------------------------------------------------------------------ more of attention's edges
@pytest.mark.parametrize("B,kv_hi,ql,hq,hkv,D,P,window", [
    (300, 200, 1, 4, 2, 64, 16, 0),        # more items than blocks, a few tokens each
    (40, 700, 1, 4, 4, 128, 16, 130),      # window shorter than the contexts
    (9, 900, 6, 4, 1, 128, 32, 0),         # 24 rows
    (9, 500, 8, 4, 1, 64, 64, 70),         # 32 rows
    (2, 5000, 1, 2, 1, 128, 64, 0)])       # one item over many blocks
def test_attention_few_rows_many_shapes(B, kv_hi, ql, hq, hkv, D, P, window):
    r = np.random.RandomState(B + kv_hi)
    kv = r.randint(0, kv_hi + 1, B).tolist()
    kv[0] = kv_hi
    lens = [ql] + r.randint(0, ql + 1, B - 1).tolist()
    pages, table, ks, vs, q, qs = make_batch(r, kv, lens, hq, hkv, D, P)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, D ** -0.5, True, window)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, D ** -0.5, True, window)
    check(out, ref, spread)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
@pytest.mark.parametrize("ql", [[1, 2], [70, 50]])
def test_attention_scale_of_any_sign(scale, ql):
    kv, hq, hkv, D, P = [140, 60], 4, 2, 64, 16
    r = np.random.RandomState(21)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    out = attend(pages, table, q, qs, kv, hq, hkv, D, P, scale)
    ok()
    ref, spread = K.attention(synth.bf16_to_f64(q), qs, ks, vs, scale)
    spread[..., 0] = abs(scale) * K.attention(synth.bf16_to_f64(q), qs, ks, vs, 1.0)[1][..., 0]
    check(out, ref, spread, norm=False)


@pytest.mark.parametrize("ql", [[3], [60]])
def test_attention_keeps_a_bad_query_to_itself(ql):
    kv, hq, hkv, D, P = [200], 2, 1, 128, 16
    r = np.random.RandomState(22)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    good = attend(pages, table, q, qs, kv, hq, hkv, D, P, 0.1)
    bad = q.copy()
    bad[1, 0, 5], bad[2, 1, 7] = 0x7FC0, 0x7F80                   # NaN, infinity
    out = attend(pages, table, bad, qs, kv, hq, hkv, D, P, 0.1)
    same = np.ones(good.shape[:2], bool)
    same[1, 0] = same[2, 1] = False
    assert np.isfinite(out[same]).all() and np.isnan(out[1, 0]).all()
    assert np.abs(out[same] - good[same]).max() <= UBF * np.abs(good).max()      # (a neighbour may rescale at another time)


def test_attention_tiles_skip_a_bad_page():
    kv, ql, hq, hkv, D, P = [300], [80], 2, 1, 64, 16
    r = np.random.RandomState(23)
    pages, table, ks, vs, q, qs = make_batch(r, kv, ql, hq, hkv, D, P)
    bad = table.copy()
    bad[0, 4] = -7
    out = attend(pages, bad, q, qs, kv, hq, hkv, D, P, 0.125)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    keep = np.r_[0:64, 80:300]
    ref, spread = np.zeros_like(out), np.zeros(out.shape[:2] + (2,))
    qf = synth.bf16_to_f64(q)
    for i in range(80):
        n = int((keep <= 220 + i).sum())
        o, s = K.attention(qf[i:i + 1], [0, 1], [ks[0][:, keep[:n]]], [vs[0][:, keep[:n]]], 0.125)
        ref[i], spread[i] = o[0], s[0]
    check(out, ref, spread)


def test_calls_replay_from_a_graph():
    """A decode step captured once and replayed as the sequence grows: lengths, pages and the cache live on the device."""
    B, hq, hkv, D, P, steps = 3, 4, 2, 64, 16, 20
    r = np.random.RandomState(24)
    start = np.array([14, 0, 31])
    cap = start + steps
    blocks = -(-cap // P)
    cache = Q.Kv4Cache.empty(int(blocks.sum()), P, hkv, D)
    table = np.full((B, int(blocks.max())), -1, np.int64)
    perm = r.permutation(cache.n_pages)
    have = -(-start // P)
    at = np.concatenate([[0], np.cumsum(have)])
    for b in range(B):
        table[b, :have[b]] = perm[at[b]:at[b + 1]]
    table_d, lens, one, nf = ints(table), ints(start), ints(np.ones(B)), ints([cache.n_pages - at[-1]])
    free = ints(perm[at[-1]:])
    qs, kl, sl, po = ints(np.zeros(B + 1)), ints(np.zeros(B)), ints(np.zeros(B)), ints(np.zeros(B))
    hist = r.randn(int(start.sum()), 2, hkv, D)
    slots = np.concatenate([table[b][np.arange(start[b]) // P] * P + np.arange(start[b]) % P for b in range(B)])
    ht = bf16_tensor(bits(hist).reshape(len(hist), -1)).view(-1, 2, hkv, D)
    Q.kv4_append(cache, ht[:, 0], ht[:, 1], ints(slots))
    k_all = [list(x) for x in np.split(K.bf16_round(hist), np.cumsum(start)[:-1])]
    x = torch.zeros((B, (hq + 2 * hkv) * D), dtype=torch.bfloat16, device="cuda")
    q, out = (torch.zeros((B, hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mk = int(cap.max())
    ws = torch.empty(Q.kv4_attention_ws_size(B, hq, hkv, D, B, 1, mk) + 1, dtype=torch.uint8, device="cuda")

    def step():
        Q.kv4_block_tables(lens, one, free, nf, P, table_d, qs, kl, sl, po, nf)
        Q.qk_norm_rope(x, hq, hkv, D, None, None, 0.0, None, None, q, None, cache=cache, slots=sl)
        Q.kv4_attention(cache, q, qs, kl, table_d, out, ws, 1, mk, D ** -0.5)
        lens.copy_(kl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            step()
    for i in range(steps):
        xs = bits(r.randn(B, hq + 2 * hkv, D))
        x.copy_(bf16_tensor(xs.reshape(B, -1)).view(torch.bfloat16))
        g.replay()
        xf = synth.bf16_to_f64(xs)
        ks, vs = [], []
        for b in range(B):
            k_all[b].append(np.stack([xf[b, hq:hq + hkv], xf[b, hq + hkv:]]))
            u, s, z = K.quantise(np.array(k_all[b]))
            d = K.dequantise(u, s, z)
            ks.append(d[:, 0].transpose(1, 0, 2))
            vs.append(d[:, 1].transpose(1, 0, 2))
        if i % 6 == 5 or i == steps - 1:
            ref, spread = K.attention(xf[:, :hq], [0, 1, 2, 3], ks, vs, D ** -0.5)
            check(out.double().cpu().numpy(), ref, spread)
    ok()
    assert lens.cpu().numpy().tolist() == cap.tolist()
