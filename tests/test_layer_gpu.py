"""The example layer: conv, delta rule and norms together, prefill and decode through a
CUDA graph.  Prefill and decode take different kernels, and q, k, v, o and the norms
are rounded to bf16 between them, so decoded rows agree with a prefill over
everything to a few bf16 steps of the largest output (2^-8 each): 8 of them."""

from __future__ import annotations

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("heads,prompts", [(2, (30, 1, 200)), (12, (700, 1, 90, 1300))])
def test_decode_continues_prefill(heads, prompts):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kda_layer

    assert kda_layer.run(heads, 3, 512, prompts) < 8 * 2.0 ** -8
