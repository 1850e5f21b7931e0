"""Host-side checks of the attention calls: what they refuse before anything is launched."""
import ctypes

import pytest

Q = pytest.importorskip("decode_matvec_gb300")
L = Q.lib()
PTR = 0x10000      # never read: every call here is refused on the host


def cache(n_pages=4, page_size=16, heads=2, dim=64, pages=PTR):
    return ctypes.byref(Q.CKv4Cache(pages, n_pages, page_size, heads, dim))


def test_page_bytes():
    assert Q.Kv4Cache.page_bytes(16, 1, 64) == 16 * 72 and Q.Kv4Cache.page_bytes(64, 8, 128) == 64 * 8 * 136


def test_workspace_size_covers_both_paths():
    few = Q.kv4_attention_ws_size(4, 8, 8, 128, 4, 1, 1000)
    many = Q.kv4_attention_ws_size(4, 8, 8, 128, 4000, 1000, 1000)
    assert 0 < few < many
    assert Q.kv4_attention_ws_size(4, 128, 1, 128, 4, 1, 1000) > 0
    for bad in ((4, 8, 3, 128, 4, 1, 10), (-1, 8, 8, 128, 4, 1, 10), (4, 8, 8, 128, -4, 1, 10), (4, 8, 8, 128, 4, 1, -1), (1 << 24, 8, 8, 64, 1, 1, 1)):
        with pytest.raises(Q.QmoeError) as e:
            Q.kv4_attention_ws_size(*bad)
        assert e.value.status == Q.QMOE_EINVAL
    for bad in ((4, 8, 8, 96, 4, 1, 10), (4, 129, 1, 64, 4, 1, 10)):
        with pytest.raises(Q.QmoeError) as e:
            Q.kv4_attention_ws_size(*bad)
        assert e.value.status == Q.QMOE_EUNSUPPORTED


@pytest.mark.parametrize("c,status", [
    (dict(page_size=8), -1), (dict(page_size=48), -1), (dict(n_pages=0), -1), (dict(heads=0), -1), (dict(pages=None), -1),
    (dict(pages=PTR + 8), -1), (dict(n_pages=1 << 27), -1), (dict(dim=96), -6)])
def test_bad_caches(c, status):
    bad = cache(**c)
    assert L.kv4_append(bad, PTR, 128, PTR, 128, 1, PTR, None) == status and Q.qmoe_last_error()
    assert L.kv4_gather(bad, PTR, 1, PTR, PTR, None) == status
    assert L.kv4_attention(bad, PTR, 1, 2, PTR, PTR, 1, PTR, 1, 1, 16, 1.0, 1, 0, PTR, PTR, 1 << 30, None) == status
    if c != dict(dim=96):
        assert L.qk_norm_rope(PTR, 512, 1, 2, 2, 64, None, None, 0.0, None, 0, 0, 0, None, PTR, None, bad, PTR, None) == status


def test_bad_arguments():
    good = cache()
    assert L.kv4_append(good, PTR, 100, PTR, 128, 2, PTR, None) == Q.QMOE_EINVAL          # stride not a multiple of 8
    assert L.kv4_append(good, PTR, 64, PTR, 128, 2, PTR, None) == Q.QMOE_EINVAL           # stride shorter than a token
    assert L.kv4_append(good, PTR + 2, 128, PTR, 128, 1, PTR, None) == Q.QMOE_EINVAL      # alignment
    assert L.kv4_append(good, PTR, 128, PTR, 128, -1, PTR, None) == Q.QMOE_EINVAL
    assert L.kv4_append(good, None, 128, PTR, 128, 1, PTR, None) == Q.QMOE_EINVAL
    assert L.kv4_gather(good, PTR, 1, None, PTR, None) == Q.QMOE_EINVAL
    att = [good, PTR, 1, 2, PTR, PTR, 1, PTR, 1, 1, 16, 1.0, 1, 0, PTR, PTR, 1 << 30, None]
    for i, v, status in ((1, None, -1), (1, PTR + 4, -1), (3, 3, -1), (4, None, -1), (6, -1, -1), (7, None, -1), (8, -1, -1),
                         (13, -5, -1), (15, None, -1), (15, PTR + 4, -1), (16, 16, -2), (3, 512, -6)):
        bad = list(att)
        bad[i] = v
        assert L.kv4_attention(*bad) == status, (i, v)
    rope = [PTR, 512, 1, 2, 2, 64, None, None, 0.0, PTR, 64, 0, 10, PTR, PTR, PTR, None, None, None]
    for i, v, status in ((0, None, -1), (1, 100, -1), (2, -1, -1), (5, 80, -6), (9, None, -1), (10, 24, -1), (10, 80, -1), (12, 0, -1),
                         (13, None, -1), (14, None, -1), (14, PTR + 2, -1), (17, PTR, -1)):
        bad = list(rope)
        bad[i] = v
        assert L.qk_norm_rope(*bad) == status, (i, v)
    tab = [PTR, PTR, 2, PTR, PTR, 16, PTR, 4, PTR, PTR, PTR, PTR, 3, PTR, None]
    for i, v in ((0, None), (2, -1), (3, None), (4, None), (5, 24), (6, None), (7, -1), (8, None), (9, None), (10, None), (12, -1), (13, None)):
        bad = list(tab)
        bad[i] = v
        assert L.kv4_block_tables(*bad) == Q.QMOE_EINVAL, (i, v)
