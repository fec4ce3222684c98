"""What the binding of the routing call refuses by itself (no GPU: it raises before the library is called)."""

import pytest
import torch

import quantized_gemm_gb300 as qg
from quantized_gemm_gb300 import build as qbuild


@pytest.mark.parametrize("shape", [(4, 3), (4, 1), (4, 8)])
def test_route_topk_refuses_indices_for_another_number_of_picks(shape):
    """The library takes the number of picks from the indices: a given tensor of another width would override k."""
    qbuild.build()
    logits = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="k is 2"):
        qg.mm_route_topk(logits, 2, indices=torch.empty(shape, dtype=torch.int32),
                         weights=torch.empty(shape, dtype=torch.float32))
