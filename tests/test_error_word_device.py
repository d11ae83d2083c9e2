"""A feed-forward block's error word has to be on the block's device (no GPU needed): the kernels set bits of
it where a call goes wrong, and a word of another GPU would make that a bad address."""
import pytest
import torch

from combine_layout_02_gb300 import experts


@pytest.mark.parametrize("checkpoint", ["bf16", "e4m3", "recompute"])
@pytest.mark.parametrize("trained", [False, True])
def test_error_word_of_another_device_is_refused(checkpoint, trained):
    x, prefix = torch.zeros(9, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    gate_up, down = torch.zeros(3, 80, 64, dtype=torch.bfloat16), torch.zeros(3, 64, 40, dtype=torch.bfloat16)
    gate_up.requires_grad_(trained)
    for dtype in (torch.int32, torch.uint32):
        with pytest.raises(ValueError, match="^all tensors have to be on the current device"):
            experts.expert_feed_forward(x, gate_up, down, prefix, checkpoint=checkpoint,
                                        err=torch.zeros(1, dtype=dtype, device="meta"))
