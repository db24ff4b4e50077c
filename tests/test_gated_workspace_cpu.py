"""The gradient's workspace around the sizes at which it changes its kernels: room for every smaller call too."""
import itertools

import pytest
import torch

import recurrent_decode_la_b200 as la
from recurrent_decode_la_b200 import build as labuild

UNITS, TOKENS = [1, 2, 3, 8, 16, 17, 31, 32, 33, 40], [1, 5, 31, 32, 33, 64, 128, 129, 300, 5000]


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 40)])
@pytest.mark.parametrize("seqs", [[0], [1, 2, 5, 16, 32, 33]])
def test_gradient_workspace_fits_smaller_calls(dtype, d, seqs):
    labuild.build()
    size = {x: la.la_gated_prefill_backward_workspace_size(dtype, 1, x[0], x[1], d, d, x[2])
            for x in itertools.product(UNITS, TOKENS, seqs)}
    for x, y in itertools.product(size, size):
        if all(a <= b for a, b in zip(x, y)):
            assert size[x] <= size[y], (x, y)
