"""KvCache on the host: it stands for the tensors it was made of (no GPU needed)."""
import pytest
import torch

import attention_backward_preprocess_gb300 as mod


def test_its_tensors_cannot_be_swapped():
    """The library holds the tensors' addresses: an attribute set to another tensor
    would be passed over, and the memory of the one before written after its end."""
    cache = mod.KvCache.__new__(mod.KvCache)
    cache._tensors = tuple(torch.full((1,), float(i)) for i in range(5))
    for i, name in enumerate(("k", "v", "k_scale", "v_scale", "block_table")):
        assert float(getattr(cache, name)) == i
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros(1))
        assert float(getattr(cache, name)) == i
