"""Shapes that no attention has are refused like any other argument (no GPU)."""
import pytest
import torch

from diffusion_transformer_denoiser_dit_b200 import attention_packed


def test_offsets_without_an_axis():
    q, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    for a, b in ((cu[0], cu), (cu, cu[0]), (cu[0], cu[0]), (cu[None], cu[None])):
        with pytest.raises(ValueError, match="cu_q and cu_k"):
            attention_packed(q, q, q, a, b, 4, 4)


def test_heads_without_features():
    q, cu = torch.zeros(4, 2, 0, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="features"):
        attention_packed(q, q, q, cu, cu, 4, 4)
