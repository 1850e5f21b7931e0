"""GPU parity with the float64 oracle: the scored router where equal values meet, every form of the row norm, and the example's steps over
chosen blocks."""
import numpy as np
import pytest

import synth
from oracle import layer as Y

from test_gpu_decoder_layer import _example
from test_gpu_kv4 import bits, check, ok
from test_gpu_layer import DEV, U32, check_norm, check_route, f64, norm_inputs, norm_tolerance

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
Q = pytest.importorskip("decode_matvec_gb300")


# ------------------------------------------------------------------ router: equal values at the border
def placed(r, T, E, rest, values):
    """Rows of `rest` with the values at random places, in every order."""
    l = np.full((T, E), float(rest))
    for t in range(T):
        l[t, r.permutation(E)[:len(values)]] = values
    return l


@pytest.mark.parametrize("E,groups", [(3, 1), (32, 1), (33, 1), (128, 4), (256, 1), (256, 8), (300, 1), (512, 1), (1024, 8), (2048, 1), (8192, 1)])
def test_route_equal_values_at_the_border_hide_no_better_one(E, groups):
    r = np.random.RandomState(E + groups)
    kw = dict(n_groups=groups, top_groups=groups, group_best=1)
    # the first two stand as one fp32 value with the third, which is larger in 64 bits alone
    l = placed(r, 24, E, -5, [20, 20, 21])
    check_route(l, 1, sigmoid=True, bias=np.zeros(E), **kw)
    check_route(l, 1, False, sigmoid=True, bias=np.full(E, 0.5), renormalise=True, **kw)
    l = placed(r, 24, E, -5, [-20, -20, -18])
    for t in range(4):
        bias = np.where(l[t] < -10, 0.5, 0.0)
        check_route(l[t:t + 1], 1, sigmoid=True, bias=bias, **kw)
        check_route(l[t:t + 1], 2, sigmoid=True, bias=bias, **kw)
        bias = np.where(l[t] < -10, 2.0, 0.0)
        check_route(l[t:t + 1], 1, bias=bias, **kw)
    # bf16 logits of two or three saturated values
    for few, p in (([20, 21], [0.9, 0.1]), ([18.5, 24, 30], [0.8, 0.15, 0.05]), ([20, 21, -np.inf], [0.4, 0.05, 0.55])):
        l = r.choice(few, (16, E), p=p)
        for k in {1, 2, min(8, E // groups), min(31, E // groups), min(32, E // groups)}:
            check_route(l, min(k, E), False, sigmoid=True, bias=np.zeros(E), **kw)
            check_route(l, min(k, E), False, sigmoid=True, bias=np.full(E, -0.75), renormalise=True, **kw)
    # scores that vanish beside their biases
    l = np.round(r.uniform(-40, -17, (16, E)))
    check_route(l, min(4, E // groups), False, sigmoid=True, bias=np.full(E, 0.25), **kw)
    l[:, 0] = 1.0
    check_route(l, min(4, E // groups), False, bias=np.where(np.arange(E) == 0, -1.0, 0.25), **kw)


@pytest.mark.parametrize("E", [3, 256, 300, 2048])
def test_route_repeated_logits_of_saturated_and_of_peaked_rows(E):
    r = np.random.RandomState(E)
    k = min(8, E - 1)
    check_route(r.uniform(12, 30, (40, E)), k, False, sigmoid=True, bias=np.zeros(E))
    l = np.round(2 * r.randn(40, E))
    l[np.arange(40), r.randint(0, E, 40)] = 60                  # one score next to 1, the others far below its rounding
    check_route(l, 1, False, bias=np.zeros(E))
    check_route(l, k, False, bias=np.zeros(E), renormalise=True)
    check_route(l, k, False, bias=np.full(E, 0.125))
    l[:] = 0.5                                                  # all the same
    check_route(l[:3], k, False, bias=np.zeros(E))
    check_route(l[:3], k, False, sigmoid=True, bias=0.5 * r.randint(0, 2, E))
    l[:, E // 2:] = -np.inf                                     # masked experts, fewer than k left
    check_route(l[:3], max(1, k), False, bias=np.zeros(E))
    check_route(l[:3], min(32, E), False, sigmoid=True, bias=np.where(np.arange(E) % 3, 0.0, -np.inf), renormalise=True)


# ------------------------------------------------------------------ router: the same logit in several warps
@pytest.mark.parametrize("E,T", [(257, 150), (300, 150), (512, 150), (1000, 100), (2048, 100), (4100, 60), (8192, 60)])
@pytest.mark.parametrize("k", [1, 2, 8, 31, 32])
def test_route_equal_logits_go_to_the_lower_expert_in_a_softmax_of_many(E, T, k):
    r = np.random.RandomState(E + k)
    l = synth.bf16_to_f64(bits(r.randn(T, E) * 2))             # bf16 logits repeat, and their largest differ from part to part
    check_route(l, k, False, bias=np.zeros(E))
    check_route(l, k, True, pad=3, bias=0.001 * r.randint(-1, 2, E), renormalise=True)
    check_route(np.round(l[:40]), k, False, bias=0.25 * r.randint(0, 2, E))


# ------------------------------------------------------------------ row norm: one to four steps a lane, one to 32 warps a row
@pytest.mark.parametrize("T,n", [(1300, 2048), (1300, 2080), (1300, 520), (1300, 1032), (1217, 4096), (2, 5136), (5, 5376), (3, 8192), (1300, 8192), (2, 16392), (3, 24584)])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_in_8_bits_of_many_and_of_wide_rows(T, n, group, f32):
    xt, x, rt, res, wt, w = norm_inputs(T, n, f32, True, n + T)
    groups, width = (-(-n // 128), 128) if group else (1, n)

    def call():
        y, out = torch.full((T, n), 3.0, dtype=torch.bfloat16, device=DEV), torch.full((T, n), 3.0, dtype=torch.bfloat16, device=DEV)
        codes, scales = torch.full((T, n), 0xAA, dtype=torch.uint8, device=DEV), torch.full((T, groups), -1.0, device=DEV)
        Q.add_rms_norm(xt, wt, 1e-5, y, residual=rt, residual_out=out, codes=codes, scales=scales)
        ok()
        return y, out, codes, scales
    y, out, codes, scales = call()
    ref = Y.add_norm(x, res, w, 1e-5)[1]
    check_norm(f64(y), ref)
    assert torch.equal(out, (xt.float() + rt.float()).to(torch.bfloat16))
    got, c = f64(scales), Y.e4m3(codes.cpu().numpy())
    s = Y.scales(ref, group)
    # the largest |y| with norm_tolerance's error, and a quotient
    assert (np.abs(got - s) <= 64 * U32 * s).all()
    unit = np.repeat(got, width, 1)[:, :n]
    # half a step of 3 fraction bits, or of the smallest step 2^-9 s; the reciprocal's and the value's own fp32 errors
    assert (np.abs(c * unit - ref) <= 2.0 ** -4 * np.abs(ref) * (1 + 2.0 ** -16) + 2.0 ** -10 * unit + norm_tolerance(ref, n)).all()
    assert all((np.abs(c[:, i:i + width]).max(1) == 448).all() for i in range(0, n, width))
    for a, b in zip(call(), (y, out, codes, scales)):          # the same bits again
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,n", [(1300, 129), (1300, 1001), (2, 1025), (3, 4096), (2, 4099), (1300, 4097)])
def test_norm_of_many_and_of_wide_rows_without_wide_loads(T, n):
    xt, x, rt, res, wt, w = norm_inputs(T, n + 1, False, True, n)          # rows begin at odd places
    y, out = (torch.full((T, n), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    Q.add_rms_norm(xt[:, 1:], wt[1:].clone(), 1e-5, y, residual=rt[:, :n], residual_out=out)
    ok()
    check_norm(f64(y), Y.add_norm(x[:, 1:], res[:, :n], w[1:], 1e-5)[1])
    assert torch.equal(out, (xt[:, 1:].float() + rt[:, :n].float()).to(torch.bfloat16))


# ------------------------------------------------------------------ as many rows as an int holds
def test_route_of_the_largest_number_of_tokens():
    T = 2 ** 31 - 1
    logits = torch.zeros((T, 1), dtype=torch.bfloat16, device=DEV)
    ids, gates = torch.full((T, 1), -9, dtype=torch.int32, device=DEV), torch.zeros((T, 1), device=DEV)
    Q.qmoe_route_scored(logits, 1, ids, gates, sigmoid=True, scale=3.0)
    ok()
    assert ids.max().item() == 0 == ids.min().item()
    assert gates.max().item() == 1.5 == gates.min().item()          # 3 / (1 + e^0)
    del logits, ids, gates
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ the example's layer for long contexts
def test_steps_attend_to_the_blocks_that_the_oracle_chooses():
    """Decode steps of the small layer, eager and replayed: the lists and the attention over them against the float64 restatement."""
    ex, top = _example(), 2
    prompts, P, hkv, D = [70, 1, 33], 16, 2, 64
    layer = ex.Layer(4, hkv, D, 4, 256, 2, n_pages=64, page_size=P, max_blocks=16, max_batch=3, top_blocks=top)
    g = torch.Generator("cuda").manual_seed(5)

    def tokens(n):
        return torch.randn((n, layer.d), generator=g, device="cuda").to(torch.bfloat16)
    ex.Step(layer, prompts, 80)(tokens(sum(prompts)))
    step, x = ex.Step(layer, [1] * 3, 80), tokens(3)

    def look():
        torch.cuda.synchronize()
        assert ex.Q.qmoe_check_status() == ex.Q.QMOE_OK
        kv, table = step.kv_len.cpu().numpy(), layer.table.cpu().numpy()
        ref = Y.select(f64(step.q), np.arange(4), kv, table, layer.bounds.codes.cpu().numpy(), f64(layer.bounds.steps), P, top, 1, 1, np.zeros((3, hkv, top), int), 80)
        assert np.array_equal(step.sel.cpu().numpy(), ref)
        check(f64(step.att), *Y.attention_blocks(f64(step.q), np.arange(4), kv, table, layer.cache.pages.cpu().numpy(), P, hkv, ref, D ** -0.5))
        return kv.tolist()
    step(x)
    assert look() == [71, 2, 34]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(x)
    torch.cuda.current_stream().wait_stream(stream)
    for i in range(4):
        x.copy_(tokens(3))
        graph.replay()
        assert look() == [72 + i, 3 + i, 35 + i]
