"""The example's layer for long contexts runs, and its attention agrees with the float64 restatement where every block is chosen."""
import pytest

from test_gpu_decoder_layer import _example

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_small_layer_that_chooses_all_blocks():
    # at most 78 tokens in pages of 16: five blocks.  The bound is that of the plain layer's test
    assert _example().main(["--small", "--top-blocks", "5"]) < 1e-2


def test_small_layer_that_chooses_some_blocks():
    # two of up to five blocks: the attention is another one, and every call succeeds
    assert _example().main(["--small", "--top-blocks", "2"]) > 1e-2
