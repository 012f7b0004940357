"""The block operators' conveniences without a GPU: what they refuse and with
which message, descriptors whose tensors change, and the package where their
extension module is missing."""
import pytest
import torch

import gemm_q4_amd as q4


@pytest.mark.parametrize("shape", [(1, 1, 16, 0), (1, 1, 0, 64), (1, 0, 16, 64), (0, 1, 16, 64)])
def test_caches_without_elements_are_refused(shape):
    """A head of no elements would be divided by in the calls that follow."""
    k = torch.zeros(shape, dtype=torch.float16)
    with pytest.raises(ValueError, match="no empty dimension"):
        q4.kv_cache(k, k.clone())
