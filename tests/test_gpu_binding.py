"""What the binding raises when a call cannot have its memory, on a GPU."""
import pytest
import torch

from linear_attention_08_b200 import kda

pytestmark = pytest.mark.gpu


def test_outputs_that_do_not_fit_raise_as_torch_does():
    """A terabyte of states: the error is the one that torch's own allocations raise."""
    cache = torch.zeros(1, 8, 128, 128, dtype=torch.int8, device="cuda")
    scales = torch.zeros(1, 8, 128, device="cuda")
    slots = torch.zeros(1 << 21, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.cuda.OutOfMemoryError):
        kda.kda_state_load(cache, scales, slots)
    assert kda.kda_state_load(cache, scales, slots[:2]).shape == (2, 8, 128, 128)
