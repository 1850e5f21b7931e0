"""GPU parity of the row norm with residual, the scored router, block bounds, block choice and attention over chosen blocks
with the float64 oracle."""
import numpy as np
import pytest

import synth
from oracle import kv4 as K
from oracle import layer as Y

from helpers import bf16_tensor
from test_gpu_kv4 import UBF, bits, check, ints, ok

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
Q = pytest.importorskip("decode_matvec_gb300")
U32 = 2.0 ** -24      # unit roundoff of fp32
DEV = "cuda"


def f64(t):
    return t.double().cpu().numpy()


def bf(x):
    """bf16 tensor of float values, and the values it holds."""
    b = bits(x)
    return bf16_tensor(b).view(torch.bfloat16), synth.bf16_to_f64(b)


# ------------------------------------------------------------------ row norm
def norm_inputs(T, n, f32, add, seed, scale=1.0):
    r = np.random.RandomState(seed)
    x = r.randn(T, n) * np.exp(r.randn(T, 1)) * scale
    if f32:
        xt = torch.from_numpy(x.astype(np.float32)).to(DEV)
        x = x.astype(np.float32).astype(np.float64)
    else:
        xt, x = bf(x)
    rt, res = bf(r.randn(T, n) * scale) if add else (None, None)
    wt, w = bf(1 + 0.3 * r.randn(n))
    return xt, x, rt, res, wt, w


def norm_tolerance(y, n):
    """What fp32 leaves of y besides its last rounding: a sum of squares in parts of at most 64 terms a thread and 10 steps of
    joining, all of one sign, halved by the root (37 U32), the addition of x and the residual (in the row's scale: it may
    cancel), and the quotient, root, eps and two products (6 U32)."""
    return (45 + 2) * U32 * np.abs(y) + 2 * U32 * np.abs(y).max(-1, keepdims=True) * 4


def check_norm(got, y):
    tol = UBF * np.abs(y) * (1 + 2.0 ** -8) + norm_tolerance(y, y.shape[1]) + 1e-38
    assert (np.abs(got - y) <= tol).all(), float((np.abs(got - y) / tol).max())


SHAPES = [(1, 1), (3, 2), (1, 7), (2, 8), (5, 129), (3, 1000), (2, 2048), (700, 2048), (33, 2080), (1000, 96), (9, 8191), (3, 8192), (2, 16392),
          (1, 32767), (2, 32768), (4097, 64)]


@pytest.mark.parametrize("T,n", SHAPES)
@pytest.mark.parametrize("f32,add", [(False, True), (True, False), (True, True)])
def test_norm(T, n, f32, add):
    xt, x, rt, res, wt, w = norm_inputs(T, n, f32, add, n + T)
    y = torch.full((T, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(y, 3.0) if add else None
    Q.add_rms_norm(xt, wt, 1e-5, y, residual=rt, residual_out=out)
    ok()
    h, ref = Y.add_norm(x, res, w, 1e-5)
    check_norm(f64(y), ref)
    if add:      # one fp32 addition, one rounding
        assert torch.equal(out, (xt.float() + rt.float()).to(torch.bfloat16))
    one = torch.empty_like(y)
    Q.add_rms_norm(xt, None, 1e-5, one, residual=rt, residual_out=out)
    check_norm(f64(one), Y.add_norm(x, res, None, 1e-5)[1])


@pytest.mark.parametrize("T,n", [(1, 8), (3, 128), (2, 136), (300, 1000), (33, 2080), (5, 4096), (2, 32768), (2000, 256)])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_in_8_bits(T, n, group):
    xt, x, rt, res, wt, w = norm_inputs(T, n, T % 2 == 0, True, n)
    y = torch.empty((T, n), dtype=torch.bfloat16, device=DEV)
    groups = -(-n // 128) if group else 1
    codes = torch.full((T, n), 0xAA, dtype=torch.uint8, device=DEV)
    scales = torch.full((T, groups), -1.0, device=DEV)
    out = torch.empty_like(y)
    Q.add_rms_norm(xt, wt, 1e-5, y, residual=rt, residual_out=out, codes=codes, scales=scales)
    ok()
    ref = Y.add_norm(x, res, w, 1e-5)[1]
    check_norm(f64(y), ref)
    s = Y.scales(ref, 128 if groups > 1 else 0)
    got = f64(scales)
    # the largest |y| with norm_tolerance's error, and a quotient
    assert (np.abs(got - s) <= 64 * U32 * s).all()
    width = 128 if groups > 1 else n
    unit = np.repeat(got, width, 1)[:, :n]
    v = Y.e4m3(codes.cpu().numpy()) * unit
    # half a step of 3 fraction bits, or of the smallest step 2^-9 s; the reciprocal's and the value's own fp32 errors
    assert (np.abs(v - ref) <= 2.0 ** -4 * np.abs(ref) * (1 + 2.0 ** -16) + 2.0 ** -10 * unit + norm_tolerance(ref, n)).all()
    # the largest value of each run has the largest code
    top = np.abs(Y.e4m3(codes.cpu().numpy()))
    assert all((top[:, i:i + width].max(1) == 448).all() for i in range(0, n, width))
    # without bf16 outputs: the same codes
    codes2, scales2 = torch.zeros_like(codes), torch.zeros_like(scales)
    Q.add_rms_norm(xt, wt, 1e-5, None, residual=rt, residual_out=out, codes=codes2, scales=scales2)
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)


@pytest.mark.parametrize("n,row,at", [(64, 96, 32), (64, 65, 0), (63, 70, 3), (2048, 2304, 256), (2048, 2051, 1)])
def test_norm_of_parts_of_rows_in_place(n, row, at):
    """Part of wider rows, in place, beside values that stay; strides and offsets with and without 16-byte alignment."""
    r = np.random.RandomState(n + row)
    T = 37
    wide, x = bf(r.randn(T + 2, row))
    wide = wide.clone()
    res, rv = bf(r.randn(T + 2, row))
    res, before_x, before_r = res.clone(), wide.clone(), res.clone()
    wt, w = bf(1 + 0.1 * r.randn(n))
    cut = slice(at, at + n)
    Q.add_rms_norm(wide[1:-1, cut], wt, 1e-6, wide[1:-1, cut], residual=res[1:-1, cut])
    ok()
    h, y = Y.add_norm(x[1:-1, cut], rv[1:-1, cut], w, 1e-6)
    check_norm(f64(wide[1:-1, cut]), y)
    assert torch.equal(res[1:-1, cut], (before_x[1:-1, cut].float() + before_r[1:-1, cut].float()).to(torch.bfloat16))
    for t, b in ((wide, before_x), (res, before_r)):
        t[1:-1, cut] = b[1:-1, cut]
        assert torch.equal(t, b)


def test_norm_of_rows_with_nothing_or_too_much():
    n, T = 256, 8
    x = torch.randn((T, n), device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] *= 1e-30
    x[4] *= 1e18
    x[5] = 0
    x[5, 3] = 2.0
    y = torch.empty((T, n), dtype=torch.bfloat16, device=DEV)
    for groups in (1, 2):
        codes, scales = torch.empty((T, n), dtype=torch.uint8, device=DEV), torch.empty((T, groups), device=DEV)
        Q.add_rms_norm(x, None, 1e-5, y, codes=codes, scales=scales)
        ok()
        got, v = f64(y), Y.e4m3(codes.cpu().numpy())
        assert not got[0].any() and not v[0].any() and not f64(scales)[0].any()
        assert np.isnan(got[1]).all() and np.isnan(f64(scales)[1]).all()
        assert np.isnan(got[2, 9]) and not np.delete(got[2], 9).any()
        # 1e-30: far below eps; 1e18: squares within fp32
        for t in (3, 4, 5, 6, 7):
            ref = Y.add_norm(f64(x[t:t + 1]), None, None, 1e-5)[1]
            check_norm(got[t:t + 1], ref)
            unit = np.repeat(f64(scales)[t:t + 1], n // groups, 1)
            assert (np.abs(v[t] * unit - ref) <= 2.0 ** -4 * np.abs(ref) * 1.001 + 2.0 ** -10 * unit + 1e-44).all()
    # scales next to fp32's smallest
    x = torch.full((1, 128), 1e-38, device=DEV)
    codes, scales = torch.empty((1, 128), dtype=torch.uint8, device=DEV), torch.empty((1, 1), device=DEV)
    Q.add_rms_norm(x, None, 1.0, y[:1, :128], codes=codes, scales=scales)
    ok()
    assert (np.abs(Y.e4m3(codes.cpu().numpy()) * f64(scales) - 1e-38) <= 1e-38 * 2.0 ** -4 + 448 * 1.5e-45).all()


# ------------------------------------------------------------------ router
def route(logits, k, f32=True, pad=0, **kw):
    T, E = logits.shape
    t = torch.from_numpy(np.ascontiguousarray(logits, dtype=np.float32)).to(DEV)
    t = t if f32 else t.to(torch.bfloat16)
    if pad:
        wide = torch.full((T, E + pad), 99.0, dtype=t.dtype, device=DEV)
        wide[:, :E] = t
        t = wide[:, :E]
    ids = torch.full((T + 1, k), -9, dtype=torch.int32, device=DEV)
    gates = torch.full((T + 1, k), -9.0, device=DEV)
    own = dict(kw)
    if own.get("bias") is not None:
        own["bias"] = torch.from_numpy(np.ascontiguousarray(own["bias"], dtype=np.float32)).to(DEV)
    Q.qmoe_route_scored(t, k, ids[:T], gates[:T], **own)
    ok()
    assert (ids[T] == -9).all() and (gates[T] == -9).all()
    return f64(t), ids[:T].cpu().numpy(), f64(gates[:T])


def check_route(logits, k, f32=True, pad=0, sigmoid=False, bias=None, n_groups=1, top_groups=1, group_best=1, renormalise=False, scale=1.0):
    seen, ids, gates = route(logits, k, f32, pad, sigmoid=sigmoid, bias=bias, n_groups=n_groups, top_groups=top_groups, group_best=group_best,
                             renormalise=renormalise, scale=scale)
    b = None if bias is None else np.asarray(bias, dtype=np.float32).astype(np.float64)
    rid, rg = Y.route(seen, k, sigmoid, b, n_groups, top_groups, group_best, renormalise, scale)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:5]
    # a logit less another (|x| U32 in the exponent, |x| <= 105 where the score is not 0), an exponential (4 U32), sums of E terms (each
    # lane's in order, then trees: E / 32 + 16), two quotients and a product; scores below fp32's normal range lose bits
    tol = (105 + 4 + logits.shape[1] / 32 + 16 + 40) * U32 * np.abs(rg) + 2.0 ** -148 * max(1.0, abs(scale))
    assert (np.abs(gates - rg) <= tol).all(), float(np.abs(gates - rg).max())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 31, 7), (4, 32, 32), (9, 33, 4), (17, 64, 8), (8, 100, 6), (40, 128, 8), (300, 256, 8), (7, 257, 9),
                                   (6, 512, 32), (5, 1000, 10), (3, 1024, 32), (4, 1025, 3), (6, 2048, 2), (2, 2049, 31), (2, 4096, 8), (2, 5000, 5), (2, 8192, 32)])
@pytest.mark.parametrize("sigmoid,biased,renorm,f32", [(False, False, False, True), (True, True, True, False), (False, True, True, True), (True, False, True, False)])
def test_route(T, E, k, sigmoid, biased, renorm, f32):
    r = np.random.RandomState(E + k)
    bias = (0.1 if sigmoid else 0.5 / E) * r.randn(E) if biased else None
    check_route(r.randn(T, E) * 2, k, f32, pad=(0, 3, 8)[E % 3], sigmoid=sigmoid, bias=bias, renormalise=renorm, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("E,groups,top,k", [(4, 2, 1, 2), (16, 4, 2, 3), (60, 4, 2, 6), (64, 8, 3, 8), (96, 3, 2, 8), (160, 8, 3, 6), (256, 8, 4, 8), (256, 32, 5, 8),
                                            (255, 15, 4, 8), (64, 32, 16, 32), (32, 32, 5, 5), (1024, 32, 4, 32), (1000, 10, 1, 8), (128, 1, 1, 8), (256, 8, 8, 8)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid,biased", [(True, True), (False, False), (False, True), (True, False)])
def test_route_groups(E, groups, top, k, best, sigmoid, biased):
    if best > E // groups:
        best = 1
    r = np.random.RandomState(E + groups + best)
    bias = (0.1 if sigmoid else 0.5 / E) * r.randn(E) if biased else None
    check_route(r.randn(40, E) * 2, k, E % 2 == 0, sigmoid=sigmoid, bias=bias, n_groups=groups, top_groups=top, group_best=best, renormalise=True)


@pytest.mark.parametrize("E,k", [(8, 3), (64, 8), (256, 8), (1024, 32), (2048, 4), (8192, 32)])
def test_route_equal_values_go_to_the_lower_expert(E, k):
    r = np.random.RandomState(E)
    few = r.randint(0, 3, (5, E)).astype(float)                # three values only
    check_route(few, k)
    check_route(few, k, sigmoid=True, bias=np.zeros(E), renormalise=True)
    check_route(few, k, False, bias=np.where(np.arange(E) % 2, 0.25, 0.5))
    check_route(np.zeros((2, E)), k, sigmoid=True, renormalise=True)
    if E <= 1024:
        for best in (1, 2):
            check_route(few, min(k, E // 4), sigmoid=True, n_groups=4, top_groups=2, group_best=best)
            check_route(few, min(k, E // 4), sigmoid=True, bias=np.zeros(E), n_groups=4, top_groups=1, group_best=best)


@pytest.mark.parametrize("E,k,groups", [(64, 8, 1), (256, 8, 8), (256, 31, 8), (512, 32, 1), (2048, 8, 1), (4500, 5, 1)])
def test_route_values_that_32_bits_cannot_tell_apart(E, k, groups):
    r = np.random.RandomState(E + 1)
    # sigmoids that 32 bits round to 1: only 64 bits order them
    check_route(r.uniform(18, 30, (6, E)), k, sigmoid=True, bias=np.zeros(E), n_groups=groups, top_groups=max(1, groups // 2), group_best=min(2, groups))
    # biases that cancel the scores up to a few units of the last place
    l = r.randn(6, E).astype(np.float32)
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    bias = (0.75 - s).astype(np.float32)
    check_route(np.repeat(l[:1], 6, 0), k, sigmoid=True, bias=bias, n_groups=groups, top_groups=max(1, groups // 2), group_best=min(2, groups))
    p = np.exp(l[0].astype(np.float64))
    p /= p.sum()
    check_route(np.repeat(l[:1], 6, 0), k, bias=(0.5 - p).astype(np.float32), n_groups=groups, top_groups=max(1, groups // 2), group_best=1)


@pytest.mark.parametrize("E,k", [(16, 4), (64, 8), (256, 8), (2048, 6)])
def test_route_masked_and_infinite_logits(E, k):
    r = np.random.RandomState(E)
    l = r.randn(9, E)
    l[0] = -np.inf                                              # nothing left
    l[1] = np.nan
    l[2, r.rand(E) < 0.9] = -np.inf
    l[3, 2:] = -np.inf                                          # fewer than k
    l[4, 3] = np.inf
    l[5] = -3.4e38                                              # a mask of the type's lowest value
    l[5, 5] = 1.0
    l[6] *= 100
    l[7] = -200 - np.arange(E) % 7                              # scores below 32 bits' range
    l[8] = 3.4e38
    for sigmoid in (False, True):
        check_route(l, k, sigmoid=sigmoid)
        for renorm in (False, True):
            check_route(l[:7], k, sigmoid=sigmoid, renormalise=renorm, bias=0.01 * r.randn(E))
        check_route(l, k, sigmoid=sigmoid, renormalise=True, scale=-1.5)
    bias = 0.1 * r.randn(E)
    bias[[1, 4]] = -np.inf                                      # experts that are off
    bias[2] = np.inf
    check_route(l[2:], k, sigmoid=True, bias=bias, renormalise=True)
    check_route(l[2:], k, sigmoid=False, bias=bias)


def test_route_agrees_with_the_plain_router():
    for T, E, k in ((9, 64, 8), (5, 2048, 2), (33, 300, 4)):
        t = torch.randn((T, E), device=DEV, generator=torch.Generator(DEV).manual_seed(E))
        a, b = (torch.empty((T, k), dtype=torch.int32, device=DEV) for _ in range(2))
        ga, gb = (torch.empty((T, k), device=DEV) for _ in range(2))
        Q.qmoe_route(t, k, a, ga)
        Q.qmoe_route_scored(t, k, b, gb)
        ok()
        assert torch.equal(a, b) and torch.allclose(ga, gb, rtol=1e-5)


# ------------------------------------------------------------------ chosen blocks
def paged(r, old, new, hkv, D, P, extra=3, scale=1.0):
    """A cache of random rows in random pages: (pages, table, kv_len, slots of the new tokens)."""
    kv = np.asarray(old) + np.asarray(new)
    blocks = -(-kv // P)
    n = int(blocks.sum()) + extra
    x = r.randn(n, hkv, 2, P, D) * scale * np.exp(0.3 * r.randn(n, hkv, 2, P, 1))
    u, s, z = K.quantise(x)
    pages = np.stack([np.concatenate([K.pack_page(u[i, h, 0], s[i, h, 0], z[i, h, 0], u[i, h, 1], s[i, h, 1], z[i, h, 1]) for h in range(hkv)])
                      for i in range(n)])
    perm = r.permutation(n)
    table = np.full((len(kv), max(1, int(blocks.max()))), -1)
    at = 0
    for b, m in enumerate(blocks):
        table[b, :m] = perm[at:at + m]
        at += m
    slots = np.concatenate([table[b, p // P] * P + p % P for b in range(len(kv)) for p in [np.arange(old[b], kv[b])]] + [np.zeros(0, int)])
    return pages, table, kv, slots.astype(np.int64)


def cache_of(pages, P, hkv, D):
    return Q.Kv4Cache(torch.from_numpy(np.ascontiguousarray(pages)).to(DEV), P, hkv, D)


@pytest.mark.parametrize("old,new,hkv,D,P", [
    ([0], [1], 1, 64, 16), ([5], [1], 2, 128, 16), ([0, 15, 16, 40], [1, 1, 1, 1], 8, 64, 16), ([0, 100], [70, 3], 3, 128, 32), ([63, 64, 0], [2, 0, 200], 4, 128, 64),
    (list(range(0, 200, 5)), [1] * 40, 4, 64, 16), ([0, 3, 0, 9, 0, 0], [900, 700, 1, 0, 33, 2000], 2, 64, 64), ([7] * 5, [1500] * 5, 16, 64, 16)])
def test_block_bounds(old, new, hkv, D, P):
    r = np.random.RandomState(sum(new) + D)
    pages, table, kv, slots = paged(r, old, new, hkv, D, P)
    slots = np.concatenate([slots, [-1, -1]])
    cache = cache_of(pages, P, hkv, D)
    b = Q.Kv4Bounds.empty(cache)
    b.codes.fill_(77)
    b.steps.fill_(-1)
    Q.kv4_block_bounds(cache, b, ints(slots))
    ok()
    codes, steps = b.codes.cpu().numpy(), f64(b.steps)
    rc, rs = np.full_like(codes, 77), np.full_like(steps, -1)
    for i in range(len(kv)):
        for j in range(old[i] // P, -(-kv[i] // P) if new[i] else 0):
            page = table[i, j]
            for h in range(hkv):
                k = K.unpack_head(pages[page].reshape(hkv, -1)[h], P, D)[0][:min(P, kv[i] - j * P)]
                rc[page, h, 0], rc[page, h, 1], rs[page, h] = Y.bounds(k)
    assert np.array_equal(codes, rc) and np.array_equal(steps, rs)


def test_block_bounds_of_extreme_rows_and_bad_slots():
    r = np.random.RandomState(4)
    P, hkv, D = 16, 1, 64
    x = np.stack([np.zeros((P, D)), np.full((P, D), 32768.0), r.randn(P, D) * 1e-7, np.where(r.rand(P, D) < 0.01, 32768.0, 1e-3 * r.randn(P, D))])
    pages = np.stack([K.pack_page(*K.quantise(k), *K.quantise(k)) for k in x])
    cache = cache_of(pages, P, hkv, D)
    b = Q.Kv4Bounds.empty(cache)
    b.codes.fill_(5)
    Q.kv4_block_bounds(cache, b, ints([15, 16 + 15, 32 + 15, 48 + 7]))
    ok()
    for i, n in enumerate((16, 16, 16, 8)):
        hi, lo, step = Y.bounds(K.unpack_head(pages[i], P, D)[0][:n])
        assert np.array_equal(b.codes[i, 0].cpu().numpy(), np.stack([hi, lo])) and float(b.steps[i, 0]) == step
    before = b.codes.clone()
    Q.kv4_block_bounds(cache, b, ints([64, -2, -1, 2 ** 31 - 1]))          # outside the cache: skipped and reported
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    assert torch.equal(before, b.codes)


def random_bounds(r, n, hkv, D):
    mid, off = 0.6 * r.randn(n, hkv, D), r.rand(n, hkv, D) + 0.3
    codes, steps = np.zeros((n, hkv, 2, D), np.int8), np.zeros((n, hkv))
    for i in range(n):
        for h in range(hkv):
            codes[i, h, 0], codes[i, h, 1], steps[i, h] = Y.bounds(np.stack([mid[i, h] + off[i, h], mid[i, h] - off[i, h]]))
    return codes, steps


def batch(r, old, new, P, extra=2):
    kv = np.asarray(old) + np.asarray(new)
    blocks = -(-kv // P)
    n = int(blocks.sum()) + extra
    perm = r.permutation(n)
    table = np.full((len(kv), max(1, int(blocks.max()))), -1)
    at = 0
    for b, m in enumerate(blocks):
        table[b, :m] = perm[at:at + m]
        at += m
    return kv, n, table, np.concatenate([[0], np.cumsum(new)])


def choose(codes, steps, q, qs, kv, table, P, top, first, last, max_kv=None, fill=-7, rows=0):
    n, hkv = q.shape[0], codes.shape[1]
    b = Q.Kv4Bounds(torch.from_numpy(codes).to(DEV), torch.from_numpy(steps.astype(np.float32)).to(DEV), P)
    sel = torch.full((n + rows, hkv, top), fill, dtype=torch.int32, device=DEV)
    max_kv = max(int(kv.max()), 0) if max_kv is None else max_kv
    size = Q.kv4_select_blocks_ws_size(n + rows, hkv, P, max_kv)
    ws = torch.full((size + 16,), 0xFF, dtype=torch.uint8, device=DEV)      # NaNs
    qt = q if rows == 0 else torch.cat([q, q[:1].expand(rows, -1, -1)])
    Q.kv4_select_blocks(b, qt, ints(qs), ints(kv), ints(table), sel, ws, max_kv, first=first, last=last)
    assert bool((ws[size:] == 0xFF).all())
    return sel.cpu().numpy()


@pytest.mark.parametrize("old,new,hq,hkv,D,P,top,first,last", [
    ([0], [1], 1, 1, 64, 16, 1, 0, 0), ([100], [1], 4, 2, 128, 16, 3, 1, 1), ([5000], [1], 16, 1, 64, 16, 64, 1, 1), ([1000, 3, 0, 333], [1, 1, 1, 1], 8, 8, 128, 32, 7, 2, 3),
    ([900, 50, 0, 0], [4, 2, 0, 5], 12, 3, 64, 64, 5, 1, 0), ([700], [3], 5, 1, 128, 16, 33, 0, 1), ([40000, 9], [1, 2], 8, 1, 64, 16, 128, 4, 8),
    ([300] * 20, [1] * 20, 40, 20, 64, 16, 6, 1, 1), ([2000], [2], 128, 1, 64, 16, 10, 3, 3), ([1500, 1501], [1, 1], 2, 2, 128, 16, 1, 0, 0), ([10], [40], 4, 2, 64, 16, 2, 1, 1),
    ([2048], [1], 66, 33, 64, 16, 100, 1, 1), ([600], [1], 4, 4, 128, 64, 4, 2, 2), ([150000], [1], 2, 1, 64, 16, 300, 1, 1)])
def test_select_blocks(old, new, hq, hkv, D, P, top, first, last):
    r = np.random.RandomState(sum(old) + top)
    kv, n, table, qs = batch(r, old, new, P)
    codes, steps = random_bounds(r, n, hkv, D)
    qt, q = bf(r.randn(int(qs[-1]), hq, D))
    got = choose(codes, steps, qt, qs, kv, table, P, top, first, last)
    ok()
    ref = Y.select(q, qs, kv, table, codes, steps, P, top, first, last, np.full(got.shape, -7), int(kv.max()))
    assert np.array_equal(got, ref)
    # larger bounds and rows of no request change nothing
    wide = choose(codes, steps, qt, qs, kv, table, P, top, first, last, max_kv=int(kv.max()) + 1000, rows=2)
    ok()
    assert np.array_equal(wide[:-2], ref) and (wide[-2:] == -7).all()


@pytest.mark.parametrize("kind", ["zero", "equal", "ties", "nan", "tiny", "huge", "negative"])
def test_select_blocks_of_special_values(kind):
    r = np.random.RandomState(8)
    P, hq, hkv, D, top = 16, 6, 2, 64, 9
    kv, n, table, qs = batch(r, [700, 90], [1, 1], P)
    codes, steps = random_bounds(r, n, hkv, D)
    q = r.randn(2, hq, D)
    if kind == "zero":
        q[:] = 0                                      # all scores 0: the lowest blocks
    if kind == "equal":
        codes[:], steps[:] = codes[0, 0], steps[0, 0]
    if kind == "ties":
        codes[:] = codes[r.randint(0, 3, n)]
        steps[:] = 0.5
    if kind == "nan":
        q[0, 1, 3], q[0, 2, 5], q[1, 5, 63] = np.nan, np.inf, -np.inf
    if kind == "tiny":
        q *= 1e-39
    if kind == "huge":
        q *= 1e38
    if kind == "negative":
        steps[:, 1] = 0
        codes[:, 0, 0] = codes[:, 0, 1] = -np.abs(codes[:, 0, 1])
        q = np.abs(q)
    qt, q = bf(q) if kind != "nan" else (torch.from_numpy(q.astype(np.float32)).to(DEV).to(torch.bfloat16), None)
    q = f64(qt) if q is None else q
    got = choose(codes, steps, qt, qs, kv, table, P, top, 1, 1)
    ok()
    assert np.array_equal(got, Y.select(q, qs, kv, table, codes, steps, P, top, 1, 1, np.full(got.shape, -7), int(kv.max())))


def test_select_blocks_reports_what_is_wrong():
    r = np.random.RandomState(9)
    P, hq, hkv, D, top = 16, 2, 1, 64, 4
    kv, n, table, qs = batch(r, [200, 100], [1, 1], P)
    codes, steps = random_bounds(r, n, hkv, D)
    qt, q = bf(r.randn(2, hq, D))
    bad = table.copy()
    bad[0, 3], bad[1, 2] = -1, n                       # blocks without a page
    got = choose(codes, steps, qt, qs, kv, bad, P, top, 1, 1)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    assert np.array_equal(got, Y.select(q, qs, kv, bad, codes, steps, P, top, 1, 1, np.full(got.shape, -7), 1000))
    got = choose(codes, steps, qt, qs, kv, table[:, :5], P, top, 1, 1)          # a table that is too narrow
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    assert np.array_equal(got, Y.select(q, qs, kv, table[:, :5], codes, steps, P, top, 1, 1, np.full(got.shape, -7), 1000))
    got = choose(codes, steps, qt, qs, kv, table, P, top, 1, 1, max_kv=150)      # a request past the bound: an empty list
    assert Q.qmoe_check_status() == Q.QMOE_ECAPACITY
    assert (got[0] == -1).all() and np.array_equal(got[1], Y.select(q, qs, kv, table, codes, steps, P, top, 1, 1, np.full(got.shape, -7), 1000)[1])
    got = choose(codes, steps, qt, qs, np.array([-3, 101]), table, P, top, 1, 1)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL and (got[0] == -1).all()
    # more queries than tokens: the first sees nothing
    got = choose(codes, steps, qt, np.array([0, 2, 2]), np.array([1, 0]), table, P, top, 1, 1)
    ok()
    assert got[:, 0].tolist() == [[-1] * 4, [0, -1, -1, -1]]


def attend(pages, table, qt, qs, kv, hkv, P, sel, scale, fill=float("nan"), rows=0, kv_list=None):
    D, hq = qt.shape[2], qt.shape[1]
    cache = cache_of(pages, P, hkv, D)
    q = qt if rows == 0 else torch.cat([qt, qt[:1].expand(rows, -1, -1)])
    s = ints(sel if rows == 0 else np.concatenate([sel] + [sel[:1]] * rows))
    out = torch.full_like(q, fill)
    size = Q.kv4_attention_blocks_ws_size(q.shape[0], hq, hkv, D, P, sel.shape[2])
    ws = torch.full((size + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    Q.kv4_attention_blocks(cache, q, ints(qs), ints(kv), ints(table), s, out, ws, scale)
    assert bool((ws[size:] == 0xFF).all())
    return f64(out)


def random_lists(r, kv, qs, P, hkv, top):
    sel = np.full((int(qs[-1]), hkv, top), -1)
    for b in range(len(kv)):
        for t in range(qs[b], qs[b + 1]):
            pos = kv[b] - (qs[b + 1] - t)
            seen = pos // P + 1 if pos >= 0 else 0
            for h in range(hkv):
                if seen <= top:
                    pick = np.arange(seen)
                else:
                    pick = np.sort(np.concatenate([[seen - 1], r.permutation(seen - 1)[:top - 1]]))
                sel[t, h, :len(pick)] = pick
    return sel


@pytest.mark.parametrize("old,new,hq,hkv,D,P,top", [
    ([0], [1], 1, 1, 64, 16, 1), ([37], [1], 4, 2, 128, 16, 2), ([500], [1], 16, 1, 64, 16, 8), ([1000, 3, 0, 333], [1, 1, 1, 1], 8, 8, 128, 32, 7),
    ([900, 50, 0, 0], [4, 2, 0, 5], 12, 3, 64, 64, 5), ([3000], [3], 5, 1, 128, 16, 60), ([2000, 9], [1, 2], 8, 1, 64, 16, 100), ([300] * 9, [1] * 9, 32, 8, 128, 64, 3),
    ([4000, 4100, 60], [1, 1, 1], 9, 1, 128, 16, 130), ([700, 800], [1, 1], 17, 1, 64, 32, 9), ([700], [2], 32, 1, 128, 16, 20), ([6000], [1], 24, 1, 128, 64, 40),
    ([20], [40], 4, 2, 64, 16, 2), ([2000] * 40, [1] * 40, 8, 8, 64, 16, 30)])
def test_attention_blocks(old, new, hq, hkv, D, P, top):
    r = np.random.RandomState(sum(old) + hq + D)
    pages, table, kv, _ = paged(r, old, new, hkv, D, P)
    qs = np.concatenate([[0], np.cumsum(new)])
    qt, q = bf(r.randn(int(qs[-1]), hq, D) * 1.5)
    sel = random_lists(r, kv, qs, P, hkv, top)
    out = attend(pages, table, qt, qs, kv, hkv, P, sel, D ** -0.5)
    ok()
    ref, spread = Y.attention_blocks(q, qs, kv, table, pages, P, hkv, sel, D ** -0.5)
    check(out, ref, spread)
    assert np.array_equal(out, attend(pages, table, qt, qs, kv, hkv, P, sel, D ** -0.5))          # the same bits again
    wide = attend(pages, table, qt, qs, kv, hkv, P, sel, D ** -0.5, fill=7.0, rows=3)
    ok()
    assert (wide[-3:] == 7).all()
    check(wide[:-3], ref, spread)


def test_attention_blocks_lists_of_all_kinds():
    """Holes, repeated blocks, blocks ahead of the query, none at all, any order."""
    r = np.random.RandomState(12)
    P, hkv, hq, D, top = 16, 1, 2, 64, 11
    old, new = [165, 165, 165, 165, 165, 165, 10], [1] * 7
    pages, table, kv, _ = paged(r, old, new, hkv, D, P)
    qs = np.arange(8)
    qt, q = bf(r.randn(7, hq, D))
    sel = np.full((7, 1, top), -1)
    sel[0, 0] = [10, -1, 3, -1, -1, 0, 9, 8, -1, 1, -1]
    sel[1, 0] = [10, 10, 2, 2, 2, 5, 5, 10, 0, 0, 10]
    sel[2, 0] = [3, 4, 11, 500, 2 ** 31 - 1, 10, 0, -1, -1, -1, -1]
    sel[4, 0] = np.arange(top)[::-1]
    sel[5, 0, 7] = 10
    sel[6, 0, 1] = 0                                             # behind the blocks that the query sees: not read
    out = attend(pages, table, qt, qs, kv, hkv, P, sel, 0.125)
    ok()
    ref, spread = Y.attention_blocks(q, qs, kv, table, pages, P, hkv, sel, 0.125)
    check(out, ref, spread, norm=False)
    assert not out[3].any() and not out[6].any() and out[5].any()
    sel[0, 0, 0], bad = -5, table.copy()
    bad[1, 5], bad[4, 9] = len(pages), -1                         # blocks without a page are not seen, and reported
    out = attend(pages, bad, qt, qs, kv, hkv, P, sel, 0.125)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    ref, spread = Y.attention_blocks(q, qs, kv, bad, pages, P, hkv, sel, 0.125)
    check(out, ref, spread, norm=False)
    out = attend(pages, table[:, :4], qt, qs, kv, hkv, P, np.maximum(sel, -1), 0.125)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL
    ref, spread = Y.attention_blocks(q, qs, kv, table[:, :4], pages, P, hkv, sel, 0.125)
    check(out, ref, spread, norm=False)
    lens = kv.copy()
    lens[2] = -1                                                  # skipped: its row stays
    out = attend(pages, table, qt, qs, lens, hkv, P, np.maximum(sel, -1), 0.125, fill=7.0)
    assert Q.qmoe_check_status() == Q.QMOE_EINVAL and (out[2] == 7).all() and (out[[0, 1, 3, 4, 5, 6]] != 7).any((1, 2)).all()


def test_attention_over_all_blocks_is_attention():
    r = np.random.RandomState(13)
    P, hkv, hq, D = 32, 2, 8, 128
    old, new = [700, 0, 64], [2, 5, 1]
    pages, table, kv, _ = paged(r, old, new, hkv, D, P)
    qs = np.concatenate([[0], np.cumsum(new)])
    qt, q = bf(r.randn(8, hq, D))
    sel = random_lists(r, kv, qs, P, hkv, 30)
    out = attend(pages, table, qt, qs, kv, hkv, P, sel, D ** -0.5)
    cache, full = cache_of(pages, P, hkv, D), torch.empty_like(qt)
    ws = torch.empty(Q.kv4_attention_ws_size(3, hq, hkv, D, 8, 5, 702), dtype=torch.uint8, device=DEV)
    Q.kv4_attention(cache, qt, ints(qs), ints(kv), ints(table), full, ws, 5, 702, D ** -0.5)
    ok()
    ref, spread = Y.attention_blocks(q, qs, kv, table, pages, P, hkv, sel, D ** -0.5)
    check(out, ref, spread)
    check(f64(full), ref, spread)


# ------------------------------------------------------------------ streams and graphs
def test_a_step_of_all_of_them_on_another_stream_and_in_a_graph():
    """Norm, cache write, bounds, choice, attention, norm, router: eager, on a side stream and replayed, the same bits; a replay
    follows the lengths and inputs that stand in its tensors."""
    g = torch.Generator(DEV).manual_seed(1)
    B, hq, hkv, D, P, top, E = 5, 8, 2, 64, 16, 6, 64
    d, width, n_pages = hq * D, (hq + 2 * hkv) * D, 200

    def w(*s):
        return torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    x0, res0, weight, w_qkv, w_r = w(B, d), w(B, d), w(d), (w(width, d) * 0.05).to(torch.bfloat16), (w(E, d) * 0.05).to(torch.bfloat16)
    bias = 0.05 * torch.randn(E, generator=g, device=DEV)
    table0 = torch.randperm(n_pages, generator=g, device=DEV)[:B * 30].int().view(B, 30).contiguous()
    lens0 = torch.tensor([0, 15, 200, 333, 470], dtype=torch.int32, device=DEV)
    kv0 = torch.randn((480, B, 2, hkv, D), generator=g, device=DEV).to(torch.bfloat16)

    def state():
        cache = Q.Kv4Cache.empty(n_pages, P, hkv, D)
        s = dict(cache=cache, bounds=Q.Kv4Bounds.empty(cache), table=table0.clone(), lens=lens0.clone(), x=x0.clone(), res=res0.clone(), new=torch.ones(B, dtype=torch.int32, device=DEV))
        for b in range(B):
            n = int(lens0[b])
            p = torch.arange(n, device=DEV)
            slots = (s["table"][b, (p // P).long()] * P + p % P).int()
            Q.kv4_append(cache, kv0[:n, b, 0], kv0[:n, b, 1], slots)
            Q.kv4_block_bounds(cache, s["bounds"], slots)
        i32 = dict(dtype=torch.int32, device=DEV)
        s.update(free=torch.zeros(1, **i32), n_free=torch.zeros(1, **i32), q_start=torch.empty(B + 1, **i32), kv_len=torch.empty(B, **i32), slots=torch.empty(B, **i32),
                 pos=torch.empty(B, **i32), y=torch.empty_like(x0), q=torch.empty((B, hq, D), dtype=torch.bfloat16, device=DEV), sel=torch.full((B, hkv, top), -9, **i32),
                 att=torch.empty((B, hq, D), dtype=torch.bfloat16, device=DEV), ids=torch.empty((B, 4), **i32), gates=torch.empty((B, 4), device=DEV),
                 codes=torch.empty((B, d), dtype=torch.float8_e4m3fn, device=DEV), scales=torch.empty((B, -(-d // 128)), device=DEV),
                 ws=torch.empty(max(Q.kv4_select_blocks_ws_size(B, hkv, P, 480), Q.kv4_attention_blocks_ws_size(B, hq, hkv, D, P, top)), dtype=torch.uint8, device=DEV))
        return s

    def step(s):
        Q.add_rms_norm(s["x"], weight, 1e-5, s["y"], residual=s["res"])
        # pages are all there: the free list stays empty unless a request begins a block
        s["q_start"].copy_(torch.arange(B + 1, dtype=torch.int32, device=DEV))
        torch.add(s["lens"], s["new"], out=s["kv_len"])
        s["pos"].copy_(s["lens"])
        s["slots"].copy_(torch.gather(s["table"], 1, (s["lens"] // P).long()[:, None])[:, 0] * P + s["lens"] % P)
        Q.qk_norm_rope(s["y"] @ w_qkv.T, hq, hkv, D, None, None, 1e-5, None, None, s["q"], cache=s["cache"], slots=s["slots"])
        Q.kv4_block_bounds(s["cache"], s["bounds"], s["slots"])
        Q.kv4_select_blocks(s["bounds"], s["q"], s["q_start"], s["kv_len"], s["table"], s["sel"], s["ws"], 480)
        Q.kv4_attention_blocks(s["cache"], s["q"], s["q_start"], s["kv_len"], s["table"], s["sel"], s["att"], s["ws"], D ** -0.5)
        Q.add_rms_norm(s["att"].view(B, d), weight, 1e-5, s["y"], residual=s["res"], codes=s["codes"], scales=s["scales"])
        Q.qmoe_route_scored(s["y"] @ w_r.T, 4, s["ids"], s["gates"], sigmoid=True, bias=bias, n_groups=4, top_groups=2, group_best=2, renormalise=True)
        s["lens"].copy_(s["kv_len"])

    def results(s):
        torch.cuda.synchronize()
        return [s[k].clone() for k in ("res", "y", "sel", "att", "ids", "gates", "scales", "lens")] + [s["codes"].view(torch.uint8).clone(), s["bounds"].codes.clone(), s["cache"].pages.clone()]

    eager = state()
    wanted = []
    for i in range(3):
        eager["x"].copy_(x0 * (i + 1))
        step(eager)
        wanted.append(results(eager))
    ok()
    # the lists against the oracle, from the state that the last step left
    codes, steps = eager["bounds"].codes.cpu().numpy(), f64(eager["bounds"].steps)
    ref = Y.select(f64(eager["q"]), np.arange(B + 1), eager["kv_len"].cpu().numpy(), eager["table"].cpu().numpy(), codes, steps, P, top, 1, 1, np.zeros((B, hkv, top), int), 480)
    assert np.array_equal(eager["sel"].cpu().numpy(), ref)
    out, spread = Y.attention_blocks(f64(eager["q"]), np.arange(B + 1), eager["kv_len"].cpu().numpy(), eager["table"].cpu().numpy(), eager["cache"].pages.cpu().numpy(), P, hkv, ref, D ** -0.5)
    check(f64(eager["att"]), out, spread)

    side = torch.cuda.Stream()
    other = state()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(3):
            other["x"].copy_(x0 * (i + 1))
            step(other)
            for a, b in zip(results(other), wanted[i]):
                assert torch.equal(a, b)
        torch.cuda.synchronize()
        held = state()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(held)
    torch.cuda.synchronize()
    for i in range(3):
        held["x"].copy_(x0 * (i + 1))
        graph.replay()
        for a, b in zip(results(held), wanted[i]):
            assert torch.equal(a, b)
    ok()


def test_calls_behind_copies_and_other_streams():
    """Each call right behind a copy of its inputs, and behind another stream's work, in a stream and in a graph: it waits for them."""
    g = torch.Generator(DEV).manual_seed(2)
    B, hq, hkv, D, P, top, E, n = 3, 4, 2, 64, 16, 3, 64, 256
    i32 = dict(dtype=torch.int32, device=DEV)
    lens = torch.tensor([100, 7, 160], **i32)
    table = torch.randperm(40, generator=g, device=DEV)[:33].int().view(B, 11).contiguous()
    q_start = torch.arange(B + 1, **i32)
    slots = (torch.gather(table, 1, ((lens - 1) // P).long()[:, None])[:, 0] * P + (lens - 1) % P).int()

    def inputs(seed):
        g = torch.Generator(DEV).manual_seed(seed)
        u = torch.randint(0, 256, (40, hkv * P * D), generator=g, device=DEV, dtype=torch.uint8)
        s = torch.stack([torch.full((40, hkv, 2 * P), 0.1, device=DEV), torch.full((40, hkv, 2 * P), -0.7, device=DEV)], -1).to(torch.float16)
        pages = torch.cat([u.view(40, hkv, P * D), s.view(torch.uint8).view(40, hkv, P * 8)], -1).reshape(40, -1).contiguous()
        return dict(x=torch.randn((700, n), generator=g, device=DEV), logits=torch.randn((600, E), generator=g, device=DEV), pages=pages,
                    q=torch.randn((B, hq, D), generator=g, device=DEV).to(torch.bfloat16), kv_len=lens.clone(), slots=slots.clone())

    def state():
        s = {k: torch.zeros_like(v) for k, v in inputs(0).items()}
        s["kv_len"].fill_(1)
        s["cache"] = Q.Kv4Cache(s["pages"], P, hkv, D)
        s.update(bounds=Q.Kv4Bounds.empty(s["cache"]), y=torch.zeros((700, n), dtype=torch.bfloat16, device=DEV), ids=torch.zeros((600, 4), **i32),
                 gates=torch.zeros((600, 4), device=DEV), sel=torch.zeros((B, hkv, top), **i32), att=torch.zeros((B, hq, D), dtype=torch.bfloat16, device=DEV),
                 ws=torch.empty(max(Q.kv4_select_blocks_ws_size(B, hkv, P, 176), Q.kv4_attention_blocks_ws_size(B, hq, hkv, D, P, top)), dtype=torch.uint8, device=DEV))
        return s

    def calls(s, src, other):
        """Copies of the inputs (each an async memory copy) with the calls right behind them; the cache's pages come by another stream."""
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            s["pages"].copy_(src["pages"])
        s["x"].copy_(src["x"])
        Q.add_rms_norm(s["x"], None, 1e-5, s["y"])
        s["logits"].copy_(src["logits"])
        Q.qmoe_route_scored(s["logits"], 4, s["ids"], s["gates"], sigmoid=True, n_groups=4, top_groups=2, group_best=2, renormalise=True)
        s["slots"].copy_(src["slots"])
        here.wait_stream(other)
        Q.kv4_block_bounds(s["cache"], s["bounds"], s["slots"])
        s["q"].copy_(src["q"])
        s["kv_len"].copy_(src["kv_len"])
        Q.kv4_select_blocks(s["bounds"], s["q"], q_start, s["kv_len"], table, s["sel"], s["ws"], 176)
        Q.kv4_attention_blocks(s["cache"], s["q"], q_start, s["kv_len"], table, s["sel"], s["att"], s["ws"], D ** -0.5)

    names = ("y", "ids", "gates", "sel", "att")
    s, src, other = state(), inputs(0), torch.cuda.Stream()
    wanted = []
    for seed in (5, 6, 7):
        for k, v in inputs(seed).items():
            src[k].copy_(v)
        torch.cuda.synchronize()
        calls(s, src, other)
        torch.cuda.synchronize()
        wanted.append([s[k].clone() for k in names] + [s["bounds"].codes.clone(), s["bounds"].steps.clone()])
        # against the oracle, for what a missing wait would show
        check_norm(f64(s["y"]), Y.add_norm(f64(src["x"]), None, None, 1e-5)[1])
        assert np.array_equal(s["ids"].cpu().numpy(), Y.route(f64(src["logits"]), 4, True, None, 4, 2, 2, True)[0])
        ref = Y.select(f64(src["q"]), np.arange(B + 1), lens.cpu().numpy(), table.cpu().numpy(), s["bounds"].codes.cpu().numpy(), f64(s["bounds"].steps), P, top, 1, 1,
                       np.zeros((B, hkv, top), int), 176)
        assert np.array_equal(s["sel"].cpu().numpy(), ref)
        check(f64(s["att"]), *Y.attention_blocks(f64(src["q"]), np.arange(B + 1), lens.cpu().numpy(), table.cpu().numpy(), src["pages"].cpu().numpy(), P, hkv, ref, D ** -0.5))
    ok()
    held, side = state(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls(held, src, other)
    torch.cuda.synchronize()
    for i, seed in enumerate((5, 6, 7)):
        for k, v in inputs(seed).items():
            src[k].copy_(v)
        torch.cuda.synchronize()
        for _ in range(3):          # (back to back: a replay begins where the one before it still ends)
            graph.replay()
        torch.cuda.synchronize()
        # the bounds' other blocks are as they were, and those that were written are the same
        for a, b in zip([held[k] for k in names], wanted[i]):
            assert torch.equal(a, b)
        page = (slots // P).long()
        assert torch.equal(held["bounds"].codes[page], wanted[i][-2][page]) and torch.equal(held["bounds"].steps[page], wanted[i][-1][page])
    ok()


# ------------------------------------------------------------------ calls at the edges of what is allowed
def test_norm_of_a_tensor_with_itself_and_of_values_that_overflow():
    r = np.random.RandomState(21)
    T, n = 5, 512
    xt, x = bf(r.randn(T, n))
    both = xt.clone()
    y = torch.empty_like(xt)
    Q.add_rms_norm(both, None, 1e-5, y, residual=both)          # x is its own residual, written in place
    ok()
    check_norm(f64(y), Y.add_norm(x, x, None, 1e-5)[1])
    assert torch.equal(both, (2 * xt.float()).to(torch.bfloat16))
    # outputs that pass fp32: the scale is infinite, finite values have code 0
    w = torch.full((n,), 3e38, dtype=torch.bfloat16, device=DEV)
    x = torch.ones((1, n), device=DEV)
    x[0, 100:] = 1e-12
    codes, scales = torch.empty((1, n), dtype=torch.uint8, device=DEV), torch.empty((1, 4), device=DEV)
    Q.add_rms_norm(x, w, 1e-30, y[:1], codes=codes, scales=scales)
    ok()
    assert np.isinf(f64(y)[0, :100]).all() and np.isfinite(f64(y)[0, 100:]).all() and np.isinf(f64(scales)[0, 0]) and np.isfinite(f64(scales)[0, 1:]).all()
    c = codes.cpu().numpy()[0]
    assert ((c[:100] & 0x7F) == 0x7F).all() and (c[100:128] & 0x7F == 0).all() and (c[128:] == 0x7E).all()


def test_route_with_biases_that_are_no_numbers():
    r = np.random.RandomState(22)
    for E in (6, 40, 300, 2048):
        bias = 0.1 * r.randn(E)
        bias[:3] = np.nan
        bias[3] = -np.inf
        k = min(E, 32)
        for sigmoid in (False, True):
            check_route(r.randn(4, E), k, sigmoid=sigmoid, bias=bias, renormalise=True)
        if E == 6:
            check_route(r.randn(4, E), 2, sigmoid=True, bias=bias, n_groups=3, top_groups=2, group_best=2)


def test_two_calls_at_once_on_two_streams():
    """The calls have no state of their own: with outputs and workspaces apart, two streams do not disturb each other."""
    r = np.random.RandomState(23)
    P, hq, hkv, D, top = 16, 8, 2, 128, 6
    sets = []
    for i in range(2):
        old, new = [900 + 50 * i, 300, 40], [1, 1, 1]
        pages, table, kv, slots = paged(r, old, new, hkv, D, P)
        qt, q = bf(r.randn(3, hq, D))
        cache = cache_of(pages, P, hkv, D)
        b = Q.Kv4Bounds.empty(cache)
        every = np.concatenate([table[j, p // P] * P + p % P for j in range(3) for p in [np.arange(kv[j])]])
        Q.kv4_block_bounds(cache, b, ints(every))
        s = dict(q=qt, cache=cache, b=b, qs=ints(np.arange(4)), kv=ints(kv), table=ints(table), sel=torch.zeros((3, hkv, top), dtype=torch.int32, device=DEV),
                 out=torch.zeros_like(qt), ws=torch.empty(1 << 20, dtype=torch.uint8, device=DEV), ws2=torch.empty(8 << 20, dtype=torch.uint8, device=DEV),
                 x=torch.randn((2000, 512), device=DEV), y=torch.zeros((2000, 512), dtype=torch.bfloat16, device=DEV), max_kv=int(kv.max()))
        s["stream"] = torch.cuda.Stream()
        sets.append(s)

    def run(s):
        Q.add_rms_norm(s["x"], None, 1e-5, s["y"])
        Q.kv4_select_blocks(s["b"], s["q"], s["qs"], s["kv"], s["table"], s["sel"], s["ws"], s["max_kv"])
        Q.kv4_attention_blocks(s["cache"], s["q"], s["qs"], s["kv"], s["table"], s["sel"], s["out"], s["ws2"], D ** -0.5)
    wanted = []
    for s in sets:
        run(s)
        torch.cuda.synchronize()
        wanted.append([s[k].clone() for k in ("y", "sel", "out")])
    for _ in range(20):
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                for k in ("y", "sel", "out"):
                    s[k].zero_()
                run(s)
    torch.cuda.synchronize()
    ok()
    for s, w in zip(sets, wanted):
        for k, v in zip(("y", "sel", "out"), w):
            assert torch.equal(s[k], v)


@pytest.mark.parametrize("n", [1, 300])
def test_calls_on_no_rows_and_on_rows_of_no_request(n):
    i32 = dict(dtype=torch.int32, device=DEV)
    cache = Q.Kv4Cache.empty(4, 16, 2, 64)
    b = Q.Kv4Bounds.empty(cache)
    q = torch.zeros((n, 4, 64), dtype=torch.bfloat16, device=DEV)
    sel, out = torch.full((n, 2, 3), -7, **i32), torch.full_like(q, 5.0)
    ws = torch.empty(8 << 20, dtype=torch.uint8, device=DEV)
    none = torch.zeros((0, 5), **i32)
    zero = torch.zeros(1, **i32)
    Q.kv4_select_blocks(b, q, zero, zero[:0], none, sel, ws, 100)                    # no requests
    Q.kv4_attention_blocks(cache, q, zero, zero[:0], none, sel, out, ws, 0.125)
    one = torch.zeros((1, 5), **i32)
    Q.kv4_select_blocks(b, q, torch.zeros(2, **i32), zero, one, sel, ws, 100)        # one, without queries
    Q.kv4_attention_blocks(cache, q, torch.zeros(2, **i32), zero, one, sel, out, ws, 0.125)
    ok()
    assert bool((sel == -7).all()) and bool((out == 5).all())
    Q.add_rms_norm(torch.zeros((0, 64), device=DEV), None, 1e-5, torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV))
    Q.qmoe_route_scored(torch.zeros((0, 64), device=DEV), 2, torch.zeros((0, 2), **i32), torch.zeros((0, 2), device=DEV))
    Q.kv4_block_bounds(cache, b, zero[:0])
    ok()


@pytest.mark.parametrize("n", [256, 264, 2048, 2080])
def test_codes_of_rows_whose_outputs_vanish(n):
    # an infinite value makes all other outputs of its row 0; so does a row without a value, or a weight of 0
    x = torch.randn((300, n), device=DEV, generator=torch.Generator(DEV).manual_seed(4))
    x[0, 9] = float("inf")
    x[1, 9] = float("nan")
    x[2] = 0
    x[3, 128:] = 0
    w = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    w[:128] = 0
    groups = (n + 127) // 128
    for weight in (None, w):
        for g in (1, groups):
            codes, scales = torch.empty((300, n), dtype=torch.uint8, device=DEV), torch.empty((300, g), device=DEV)
            Q.add_rms_norm(x, weight, 1e-5, codes=codes, scales=scales)
            ok()
            c, s = codes.cpu().numpy() & 0x7F, f64(scales)
            if g == 1:
                assert (c[0] == 0x7F).all() and np.isnan(s[0]).all()
            else:
                assert (c[0, :128] == 0x7F).all() and np.isnan(s[0, 0]) and not c[0, 128:].any() and not s[0, 1:].any()
                assert not c[3, 128:].any() and not s[3, 1:].any()
                if weight is not None:
                    assert not c[4:, :128].any() and not s[4:, 0].any()
            assert (c[1] == 0x7F).all() and np.isnan(s[1]).all() and not c[2].any() and not s[2].any()
            assert ((c[4:].reshape(296, -1) == 0x7E).any(1)).all() and not (c[4:] == 0x7F).any()


@pytest.mark.parametrize("B,n_kv,page,lens,top", [
    (3, 1, 16, 8000, 33), (40, 8, 16, 2100, 9), (2, 2, 16, 8190, 300), (1, 1, 16, 120000, 128), (2, 1, 16, 33000, 40), (45, 8, 64, 32000, 64),
    (1, 1, 16, 200000, 64), (2, 1, 16, 300000, 9000)])
def test_select_blocks_by_every_split_of_a_list(B, n_kv, page, lens, top):
    # lists of few distinct scores (whole tiers of equal ones at the last place taken), of distinct ones, and of one score alone
    r = np.random.RandomState(B + page + top)
    D, blocks = 64, (lens + page - 1) // page
    n_pages = max(512, blocks)
    table = np.stack([r.permutation(n_pages)[:blocks] for _ in range(B)]).astype(np.int32)
    kv = r.randint(lens // 2, lens + 1, B).astype(np.int32)
    kv[0] = lens
    q = r.randn(B, n_kv, D)
    qt, q = bf(q)
    for kind in range(3):
        codes = r.randint(-127, 128, (n_pages, n_kv, 2, D)) if kind < 2 else np.ones((n_pages, n_kv, 2, D))
        if kind == 1:
            codes[:] = codes[:3][r.randint(0, 3, n_pages)]
        codes = np.sort(codes, 2)[:, :, ::-1].astype(np.int8)
        steps = np.full((n_pages, n_kv), 0.125, np.float32)
        bounds = Q.Kv4Bounds(torch.tensor(codes.copy(), device=DEV), torch.tensor(steps, device=DEV), page)
        ws = torch.empty(Q.kv4_select_blocks_ws_size(B, n_kv, page, lens), dtype=torch.uint8, device=DEV)
        sel = torch.full((B, n_kv, top), -7, dtype=torch.int32, device=DEV)
        Q.kv4_select_blocks(bounds, qt, torch.arange(B + 1, dtype=torch.int32, device=DEV), torch.tensor(kv, device=DEV),
                            torch.tensor(table, device=DEV), sel, ws, lens)
        ok()
        want = Y.select(q, np.arange(B + 1), kv, table, codes, steps, page, top, 1, 1, np.full((B, n_kv, top), -7), lens)
        assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [7, 256, 2000])
def test_renormalised_gate_of_one_expert_is_the_scale(E, sigmoid):
    logits = 30 * torch.randn((777, E), device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    ids, gates = torch.empty((777, 1), dtype=torch.int32, device=DEV), torch.empty((777, 1), device=DEV)
    Q.qmoe_route_scored(logits, 1, ids, gates, sigmoid=sigmoid, renormalise=True, scale=2.5)
    ok()
    assert torch.equal(ids[:, 0].long(), logits.argmax(1)) and bool((gates == 2.5).all())
