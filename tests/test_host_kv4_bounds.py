"""Host-side properties of the attention calls beyond what they refuse: sizes and argument checks of the Python binding."""
import itertools

import pytest

Q = pytest.importorskip("decode_matvec_gb300")


@pytest.mark.parametrize("group,dim", [(g, d) for g in (1, 2, 3, 4, 5, 7, 8, 16, 31, 32, 33, 128) for d in (64, 128)])
def test_workspace_for_the_largest_call_serves_the_others(group, dim):
    """The size does not fall when the batch, the tokens or the longest query grow."""
    Bs, tokens, longest = (0, 1, 2, 64, 1000), (0, 1, 7, 40, 300, 5000), tuple(range(40)) + (64, 100, 2048)
    size = {c: Q.kv4_attention_ws_size(c[0], 2 * group, 2, dim, c[1], c[2], 1000) for c in itertools.product(Bs, tokens, longest)}
    for B, n, q in size:
        for bigger in ((x, n, q) for x in Bs if x > B), ((B, x, q) for x in tokens if x > n), ((B, n, x) for x in longest if x > q):
            for c in bigger:
                assert size[B, n, q] <= size[c], ((B, n, q), c)


# ------------------------------------------------------------------ types and devices of tensors
torch = pytest.importorskip("torch")


class OnDevice:
    """A host tensor that says it is on cuda:`index`: for checks alone, its pointer is never read."""

    def __init__(self, t, index=0):
        self.t, self.index, self.is_cuda = t, index, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


#: call -> its tensors by argument name (two requests or tokens, two kv heads of 64, pages of 16)
TENSORS = dict(
    kv4_block_tables=dict(cached=i32(2), new_tokens=i32(2), free_pages=i32(4), n_free=i32(1), table=i32(2, 3), q_start=i32(3),
                          kv_len=i32(2), slots=i32(2), positions=i32(2), n_free_out=i32(1)),
    qk_norm_rope=dict(qkv=bf16(2, 8 * 64), q_weight=bf16(64), k_weight=bf16(64), cos_sin=torch.zeros(10, 64), positions=i32(2),
                      q_out=bf16(2, 4, 64), k_out=bf16(2, 2, 64), slots=i32(2)),
    kv4_append=dict(k=bf16(2, 2, 64), v=bf16(2, 2, 64), slots=i32(2)),
    kv4_gather=dict(slots=i32(2), k_out=bf16(2, 2, 64), v_out=bf16(2, 2, 64)),
    kv4_attention=dict(q=bf16(2, 4, 64), q_start=i32(3), kv_len=i32(2), table=i32(2, 3), out=bf16(2, 4, 64),
                       workspace=torch.zeros(4096, dtype=torch.uint8)))
NUMBERS = dict(kv4_block_tables=dict(page_size=16), qk_norm_rope=dict(n_q_heads=4, n_kv_heads=2, head_dim=64, eps=1e-5),
               kv4_append={}, kv4_gather={}, kv4_attention=dict(max_q=1, max_kv=16, scale=0.125))


@pytest.fixture
def call(monkeypatch):
    """Makes a call on the named tensors (device 0 is current); returns whether it got as far as the library."""
    reached = []
    monkeypatch.setattr(Q, "_raw_stream", (lambda: 0, lambda device: 0))
    for name in [*TENSORS, "kv4_block_tables_bounded"]:
        monkeypatch.setattr(Q._lib, name, lambda *a: reached.append(a) or 0)
    pages = OnDevice(torch.zeros((4, Q.Kv4Cache.page_bytes(16, 2, 64)), dtype=torch.uint8))

    def run(name, pages=pages, **other):
        cache = {} if name == "kv4_block_tables" else dict(cache=Q.Kv4Cache(pages, 16, 2, 64))
        del reached[:]
        getattr(Q, name)(**cache, **NUMBERS[name], **{k: OnDevice(v) for k, v in TENSORS[name].items()} | other)
        return bool(reached)
    run.reached, run.undo = reached, monkeypatch.undo
    return run


@pytest.mark.parametrize("name", TENSORS)
def test_right_tensors_reach_the_library(call, name):
    assert call(name)
    for arg, t in TENSORS[name].items():
        if t.dtype == torch.bfloat16:                       # bf16 bits in integers are bf16
            assert call(name, **{arg: OnDevice(t.view(torch.int16))})


@pytest.mark.parametrize("name,arg", [(n, a) for n in TENSORS for a in TENSORS[n]])
def test_wrong_types_and_places_are_refused(call, name, arg):
    t = TENSORS[name][arg]
    wrong = [t] if t.dtype == torch.uint8 else []                                # host memory
    wrong += [OnDevice(t, 1)]                                                     # another GPU's
    if t.dtype == torch.bfloat16:
        wrong += [OnDevice(t.half())]                                             # as wide
    elif t.dtype == torch.int32:
        wrong += [OnDevice(t.float()), OnDevice(t.long())]
    elif t.dtype == torch.float32:
        wrong += [OnDevice(t.int()), OnDevice(t.half())]
    for w in wrong + [t]:
        with pytest.raises(ValueError):
            call(name, **{arg: w})
        assert not call.reached


@pytest.mark.parametrize("name", [n for n in TENSORS if n != "kv4_block_tables"])
def test_caches_elsewhere_are_refused(call, name):
    pages = torch.zeros((4, Q.Kv4Cache.page_bytes(16, 2, 64)), dtype=torch.uint8)
    for p in (pages, OnDevice(pages, 1)):
        with pytest.raises(ValueError):
            call(name, pages=p)
        assert not call.reached


def test_block_tables_hand_the_library_the_size_of_the_stack(call):
    call("kv4_block_tables")
    assert call.reached[0][4] == TENSORS["kv4_block_tables"]["free_pages"].numel()
    L, ptr = Q.lib(), 0x10000      # (never read: refused on the host)
    tab = [ptr, ptr, 2, ptr, -1, ptr, 16, ptr, 4, ptr, ptr, ptr, ptr, 3, ptr, None]
    call.undo()
    assert L.kv4_block_tables_bounded(*tab) == Q.QMOE_EINVAL
