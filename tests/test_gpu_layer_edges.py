"""GPU parity of the scored router with the float64 oracle where equal values meet."""
import numpy as np
import pytest

import synth

from test_gpu_kv4 import bits
from test_gpu_layer import check_route

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


# ------------------------------------------------------------------ router: the same logit in several warps
@pytest.mark.parametrize("E,T", [(257, 150), (300, 150), (512, 150), (1000, 100), (2048, 100), (4100, 60), (8192, 60)])
@pytest.mark.parametrize("k", [1, 2, 8, 31, 32])
def test_route_equal_logits_go_to_the_lower_expert_in_a_softmax_of_many(E, T, k):
    r = np.random.RandomState(E + k)
    l = synth.bf16_to_f64(bits(r.randn(T, E) * 2))             # bf16 logits repeat, and their largest differ from part to part
    check_route(l, k, False, bias=np.zeros(E))
    check_route(l, k, True, pad=3, bias=0.001 * r.randint(-1, 2, E), renormalise=True)
    check_route(np.round(l[:40]), k, False, bias=0.25 * r.randint(0, 2, E))
