"""The status word of the packed-layer calls is written by the device as one int32: nothing else is taken (no GPU)."""
import pytest
import torch

from diffusion_transformer_denoiser_dit_b200 import attention_packed, linear_fused

BAD = [torch.zeros(1), torch.zeros(1, dtype=torch.int64), torch.zeros(4, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32),
       torch.zeros(1, dtype=torch.int16)]


@pytest.mark.parametrize("status", BAD, ids=lambda t: f"{t.dtype}-{t.numel()}")
def test_status_is_an_int32(status):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="status"):
        linear_fused(x, w, status=status)
    q, cu = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="status"):
        attention_packed(q, q, q, cu, cu, 4, 4, status=status)
