"""Host-side checks of the row norm, the scored router and the calls over chosen blocks: what they refuse before anything
is launched."""
import ctypes

import pytest

Q = pytest.importorskip("decode_matvec_gb300")
torch = pytest.importorskip("torch")
from test_host_kv4_bounds import OnDevice, bf16, i32  # noqa: E402

L = Q.lib()
PTR = 0x10000      # never read: every call here is refused on the host


def refused(f, good, changes):
    for i, v, status in changes:
        bad = list(good)
        bad[i] = v
        assert f(*bad) == status, (i, v)
        assert Q.qmoe_last_error()


def cache(n_pages=4, page_size=16, heads=2, dim=64, pages=PTR):
    return ctypes.byref(Q.CKv4Cache(pages, n_pages, page_size, heads, dim))


def bounds(n_pages=4, page_size=16, heads=2, dim=64, codes=PTR, steps=PTR):
    return ctypes.byref(Q.CKv4Bounds(codes, steps, n_pages, page_size, heads, dim))


def test_norm():
    good = [PTR, 0, 64, PTR, 64, PTR, 64, PTR, 2, 64, 1e-5, PTR, 64, PTR, PTR, 128, None]
    refused(L.add_rms_norm, good, [
        (0, None, -1), (0, PTR + 1, -1), (2, 63, -1), (3, None, -1), (4, 60, -1), (5, None, -1), (6, 60, -1), (7, PTR + 1, -1),
        (8, -1, -1), (9, 0, -1), (9, 32769, -1), (10, 0.0, -1), (10, -1.0, -1), (10, float("nan"), -1), (10, float("inf"), -1),
        (11, PTR + 1, -1), (12, 60, -1), (13, None, -1), (14, None, -1), (14, PTR + 2, -1), (15, 64, -6),
        # codes want whole groups of eight
        (0, PTR + 2, -6), (2, 65, -6), (9, 63, -6), (13, PTR + 4, -6), (3, PTR + 2, -6), (11, PTR + 8, -6)])
    none = list(good)
    none[11] = none[13] = none[14] = None
    assert L.add_rms_norm(*none) == -1
    f32 = list(good)
    f32[1], f32[0] = 1, PTR + 2
    assert L.add_rms_norm(*f32) == -1


def test_route():
    good = [PTR, 1, 64, 2, 64, 8, 1, PTR, 8, 4, 2, 1, 1.0, PTR, PTR, None]
    refused(L.qmoe_route_scored, good, [
        (0, None, -1), (0, PTR + 2, -1), (2, 63, -1), (3, -1, -1), (4, 0, -1), (4, 8193, -1), (5, 0, -1), (5, 33, -1), (5, 65, -1),
        (6, 2, -1), (6, -1, -1), (7, PTR + 2, -1), (8, 0, -1), (8, 7, -1), (8, 64, -1), (9, 0, -1), (9, 9, -1), (10, 0, -1), (10, 3, -1),
        (12, float("nan"), -1), (12, float("inf"), -1), (13, None, -1), (14, None, -1), (13, PTR + 2, -1), (14, PTR + 1, -1)])
    few = list(good)
    few[8], few[9], few[10] = 32, 3, 2                          # 3 groups of 2 experts cannot give 8
    assert L.qmoe_route_scored(*few) == -1
    one = list(good)
    one[4], one[5], one[8], one[9] = 32, 2, 32, 32              # groups of one expert have no best two
    assert L.qmoe_route_scored(*one) == -1
    wide = list(good)
    wide[2], wide[4] = 2048, 2048
    assert L.qmoe_route_scored(*wide) == -6


def test_chosen_blocks():
    refused(L.kv4_block_bounds, [cache(), bounds(), PTR, 3, None], [
        (0, cache(page_size=8), -1), (0, cache(pages=None), -1), (0, cache(dim=96), -6), (1, None, -1), (1, bounds(codes=None), -1),
        (1, bounds(steps=None), -1), (1, bounds(codes=PTR + 8), -1), (1, bounds(steps=PTR + 2), -1), (1, bounds(n_pages=5), -1),
        (1, bounds(page_size=32), -1), (1, bounds(heads=1), -1), (1, bounds(dim=128), -1), (2, None, -1), (3, -1, -1)])
    sel = [bounds(), PTR, 3, 4, PTR, PTR, 2, PTR, 5, 100, 4, 1, 1, PTR, PTR, 1 << 20, None]
    refused(L.kv4_select_blocks, sel, [
        (0, None, -1), (0, bounds(page_size=24), -1), (0, bounds(dim=80), -6), (0, bounds(heads=0), -1), (0, bounds(n_pages=1 << 27), -1),
        (1, None, -1), (1, PTR + 8, -1), (2, -1, -1), (3, 3, -1), (3, 1, -1), (3, 258, -6), (4, None, -1), (5, None, -1), (6, -1, -1),
        (7, None, -1), (8, -1, -1), (9, -1, -1), (9, 0x7FFFFFFF, -1), (10, 0, -1), (10, 65537, -1), (11, -1, -1), (12, -1, -1),
        (11, 4, -1), (13, None, -1), (14, None, -1), (14, PTR + 4, -1), (15, 10, -2), (2, 0x7FFFFFFF, -2)])
    att = [cache(), PTR, 3, 4, PTR, PTR, 2, PTR, 5, PTR, 4, 0.1, PTR, PTR, 1 << 30, None]
    refused(L.kv4_attention_blocks, att, [
        (0, None, -1), (0, cache(page_size=24), -1), (0, cache(dim=80), -6), (1, None, -1), (1, PTR + 8, -1), (2, -1, -1), (3, 3, -1),
        (3, 1, -1), (3, 66, -6), (4, None, -1), (5, None, -1), (6, -1, -1), (7, None, -1), (8, -1, -1), (9, None, -1), (10, 0, -1),
        (10, 65537, -1), (12, None, -1), (12, PTR + 2, -1), (13, None, -1), (13, PTR + 4, -1), (14, 100, -2), (2, 0x7FFFFFFF, -1)])


def test_nothing_to_do_is_no_error():
    assert L.add_rms_norm(None, 0, 64, None, 0, None, 0, None, 0, 64, 1e-5, None, 64, None, None, 0, None) == 0
    assert L.qmoe_route_scored(None, 1, 64, 0, 64, 8, 1, None, 1, 1, 1, 1, 1.0, None, None, None) == 0
    assert L.kv4_block_bounds(cache(), bounds(), None, 0, None) == 0
    assert L.kv4_select_blocks(bounds(), None, 0, 4, None, None, 0, None, 0, 100, 4, 1, 1, None, None, 0, None) == 0
    assert L.kv4_attention_blocks(cache(), None, 0, 4, None, None, 0, None, 0, None, 4, 0.1, None, None, 0, None) == 0


def test_workspace_sizes():
    size = Q.kv4_select_blocks_ws_size
    assert size(3, 2, 16, 100) >= 3 * 2 * 7 * 4 and size(0, 2, 16, 100) == 0
    for n in (1, 2, 50):
        for kv in (0, 1, 99, 5000):
            assert size(n, 2, 16, kv) <= size(n + 1, 2, 16, kv) and size(n, 2, 16, kv) <= size(n, 2, 16, kv + 17)
    for bad in ((-1, 2, 16, 10), (1, 0, 16, 10), (1, 2, 8, 10), (1, 2, 16, -1)):
        with pytest.raises(Q.QmoeError):
            size(*bad)
    size = Q.kv4_attention_blocks_ws_size
    for G in (1, 4, 8, 9, 17, 32):
        for D in (64, 128):
            sizes = [size(n, 2 * G, 2, D, 16, t) for n in (1, 3, 900) for t in (1, 9, 600)]
            assert min(sizes) > 0 and size(900, 2 * G, 2, D, 16, 600) == max(sizes)
    for bad, status in (((-1, 4, 2, 64, 16, 4), -1), ((1, 3, 2, 64, 16, 4), -1), ((1, 4, 2, 64, 16, 0), -1), ((1, 4, 2, 64, 8, 4), -1), ((1, 66, 2, 64, 16, 4), -6)):
        with pytest.raises(Q.QmoeError) as e:
            size(*bad)
        assert e.value.status == status


# ------------------------------------------------------------------ types and devices of tensors
def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


TENSORS = dict(
    add_rms_norm=dict(x=bf16(2, 256), weight=bf16(256), y=bf16(2, 256), residual=bf16(2, 256), residual_out=bf16(2, 256),
                      codes=torch.zeros((2, 256), dtype=torch.uint8), scales=f32(2, 2)),
    qmoe_route_scored=dict(logits=bf16(2, 16), ids=i32(2, 3), gates=f32(2, 3), bias=f32(16)),
    kv4_block_bounds=dict(slots=i32(2)),
    kv4_select_blocks=dict(q=bf16(2, 4, 64), q_start=i32(3), kv_len=i32(2), table=i32(2, 3), sel=i32(2, 2, 4),
                           workspace=torch.zeros(4096, dtype=torch.uint8)),
    kv4_attention_blocks=dict(q=bf16(2, 4, 64), q_start=i32(3), kv_len=i32(2), table=i32(2, 3), sel=i32(2, 2, 4), out=bf16(2, 4, 64),
                              workspace=torch.zeros(4096, dtype=torch.uint8)))
NUMBERS = dict(add_rms_norm=dict(eps=1e-5), qmoe_route_scored=dict(k=3), kv4_block_bounds={}, kv4_select_blocks=dict(max_kv=48),
               kv4_attention_blocks=dict(scale=0.125))


@pytest.fixture
def call(monkeypatch):
    """Makes a call on the named tensors (device 0 is current); returns whether it got as far as the library."""
    reached = []
    monkeypatch.setattr(Q, "_raw_stream", (lambda: 0, lambda device: 0))
    for name in TENSORS:
        monkeypatch.setattr(Q._lib, name, lambda *a: reached.append(a) or 0)

    def run(name, index=0, **other):
        pages = OnDevice(torch.zeros((4, Q.Kv4Cache.page_bytes(16, 2, 64)), dtype=torch.uint8), index)
        b = Q.Kv4Bounds(OnDevice(torch.zeros((4, 2, 2, 64), dtype=torch.int8), index), OnDevice(f32(4, 2), index), 16)
        own = {} if not name.startswith("kv4") else dict(bounds=b) if name == "kv4_select_blocks" else dict(cache=Q.Kv4Cache(pages, 16, 2, 64))
        if name == "kv4_block_bounds":
            own["bounds"] = b
        del reached[:]
        getattr(Q, name)(**own, **NUMBERS[name], **{k: OnDevice(v) for k, v in TENSORS[name].items()} | other)
        return bool(reached)
    run.reached = reached
    return run


@pytest.mark.parametrize("name", TENSORS)
def test_right_tensors_reach_the_library(call, name):
    assert call(name)
    for arg, t in TENSORS[name].items():
        if t.dtype == torch.bfloat16:                       # bf16 bits in integers are bf16
            assert call(name, **{arg: OnDevice(t.view(torch.int16))})


@pytest.mark.parametrize("name,arg", [(n, a) for n in TENSORS for a in TENSORS[n]])
def test_wrong_types_places_and_shapes_are_refused(call, name, arg):
    t = TENSORS[name][arg]
    wrong = [t, OnDevice(t, 1)]                                                   # host memory, another GPU's
    if arg not in ("workspace",):
        wrong += [OnDevice(t.to(torch.float64)), OnDevice(t.half() if t.dtype != torch.float32 else t.int())]
        wrong += [OnDevice(t[:1])] if arg not in ("table", "weight", "bias") else []
    if arg in ("weight", "bias", "y", "gates", "codes", "scales", "sel", "out"):
        wrong += [OnDevice(torch.cat([t, t], -1)[..., :-1])]
    if arg in ("x", "y", "residual", "residual_out", "logits"):
        wrong += [OnDevice(torch.stack([t, t], -1)[..., 0])]                      # every other value
    if arg in ("ids", "codes", "scales", "q", "sel", "out"):
        wrong += [OnDevice(torch.cat([t, t], -1)[..., :t.shape[-1]])]             # rows apart
    if arg == "slots":
        wrong = [t, OnDevice(t, 1), OnDevice(t.long())]
    for w in wrong:
        with pytest.raises((ValueError, RuntimeError)):
            call(name, **{arg: w})
        assert not call.reached


@pytest.mark.parametrize("name", [n for n in TENSORS if n.startswith("kv4")])
def test_handles_elsewhere_are_refused(call, name):
    with pytest.raises(ValueError):
        call(name, index=1)
    assert not call.reached


def test_scales_without_codes_and_outputs_without_inputs_are_refused(call):
    t = {k: OnDevice(v) for k, v in TENSORS["add_rms_norm"].items()}
    for drop in ("codes", "scales", "residual"):
        with pytest.raises(ValueError):
            Q.add_rms_norm(eps=1e-5, **{k: v for k, v in t.items() if k != drop})
        assert not call.reached
    Q.add_rms_norm(eps=1e-5, **{k: v for k, v in t.items() if k in ("x", "y")}, weight=None)
    assert call.reached


def test_bounds_handles():
    good = dict(codes=OnDevice(torch.zeros((4, 2, 2, 64), dtype=torch.int8)), steps=OnDevice(f32(4, 2)), page_size=16)
    Q.Kv4Bounds(**good)
    for bad in (dict(codes=OnDevice(torch.zeros((4, 2, 2, 64), dtype=torch.uint8))), dict(codes=OnDevice(torch.zeros((4, 2, 64), dtype=torch.int8))),
                dict(codes=OnDevice(torch.zeros((4, 2, 3, 64), dtype=torch.int8))), dict(steps=OnDevice(f32(4, 3))), dict(steps=OnDevice(f32(4, 2).double())),
                dict(steps=OnDevice(f32(4, 2), 1)), dict(steps=OnDevice(f32(2, 4).t()))):
        with pytest.raises(ValueError):
            Q.Kv4Bounds(**{**good, **bad})
