"""The attention-block example end to end: quantized QKV and O products around
the 4-bit cache, prompts, then decoding steps from a graph."""
import pytest

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,window", [(4, 0), (8, 100)])
def test_attention_block(bits, window):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import attention_block
    gu.announce("attention block, W%dA8, window %d" % (bits, window))
    r = attention_block.main(["--batch", "3", "--prompt", "150", "--steps", "8", "--bits", str(bits),
                              "--window", str(window)])
    assert r["finite"]
    if window == 0:
        # absmax int4 groups of 64 normal values: a code's step is 2.5 / 7 of the standard deviation, so keys and
        # values are off by a step / sqrt(12), about a tenth each; the averages over tokens stay of that order
        assert 0.02 < r["error"] < 0.3
