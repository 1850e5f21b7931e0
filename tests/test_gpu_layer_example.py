"""The example's layer for long contexts runs, and its attention agrees with the float64 restatement where every block is chosen."""
import numpy as np
import pytest

from oracle import layer as Y

from test_gpu_decoder_layer import _example
from test_gpu_kv4 import check
from test_gpu_layer import f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_small_layer_that_chooses_all_blocks():
    # at most 78 tokens in pages of 16: five blocks.  The bound is that of the plain layer's test
    assert _example().main(["--small", "--top-blocks", "5"]) < 1e-2


def test_small_layer_that_chooses_some_blocks():
    # two of up to five blocks: the attention is another one, and every call succeeds
    assert _example().main(["--small", "--top-blocks", "2"]) > 1e-2


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
