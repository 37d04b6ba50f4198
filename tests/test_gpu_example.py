"""The decode example: quantized projections, cache and attention together,
captured in a graph and replayed, against binary32 on the same packed data."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("bits,dtype", [(4, "f16"), (8, "bf16"), (16, "f16")])
def test_decode_step(tokens, bits, dtype):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_step
    kind = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    off, _ = decode_step.generate(tokens=tokens, cache_bits=bits, dtype=kind, steps=4)
    # q, the attention's output, both projections and y are each rounded to 11
    # or 8 bits: five roundings of at most 2^-11 or 2^-8, the sums over 512
    # terms of random sign grow slower than their largest value
    assert off < 5 * {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype] * 4
