"""The example of a decoder layer's attention: prompt chunks, a verified tree of drafts and decoding after it agree with one
prompt.  Both paths see the same cached values; q|k|v rows come from batches of other sizes (bounded by 1e-3 of sum |x w| each
against the definition, in practice by fp32 sums in another order), the attention's outputs are fp16: 2^-10 of them each side,
which the o product averages.  1% of the rms of what the attention adds leaves
room for all of that.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.late]
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_attention.py")


@pytest.mark.parametrize("cache", ["f16", "int8", "q4_0"])
def test_drafts_agree_with_a_prompt(cache):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from bit_weight_only_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decoder_attention", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    off, rms = example.run(cache)
    assert off <= 0.01 * rms
