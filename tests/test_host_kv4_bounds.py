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
