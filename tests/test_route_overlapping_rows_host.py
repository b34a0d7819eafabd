"""Host-side checks (no GPU needed) of router logits whose rows overlap: a row stride below the number of experts
is refused by the call, and a helper that hid it would have the kernel read past the tensor."""
import pytest
import torch

import nvfp4_quantized_linear_gb300 as nv


@pytest.mark.parametrize("logits", [
    torch.zeros(32).expand(1000, 32),                        # one row for all tokens
    torch.zeros(130).as_strided((50, 32), (2, 1)),           # a sliding window
    torch.zeros(63, dtype=torch.bfloat16).as_strided((2, 32), (31, 1))])
def test_overlapping_rows_are_refused(logits):
    tokens = logits.shape[0]
    with pytest.raises(ValueError, match="^logits has overlapping rows"):
        nv.moe_route(logits, 4)
    ids, dw = torch.zeros(tokens, 4, dtype=torch.int32), torch.zeros(tokens, 4)
    with pytest.raises(ValueError, match="^logits has overlapping rows"):
        nv.moe_route_backward(dw, ids, logits)


@pytest.mark.parametrize("logits", [torch.zeros(32).expand(1, 32), torch.zeros(32)[None], torch.zeros(0, 32),
                                    torch.zeros(64).as_strided((1, 32), (5, 1)), torch.zeros(9, 40)[:, 5:37]])
def test_other_strides_are_taken(logits):
    """One row or none has no stride that matters; these get as far as the check of the device."""
    with pytest.raises(ValueError, match="^logits must be a CUDA"):
        nv.moe_route(logits, 4)
