"""What the binding raises on a GPU: errors of this call, as PyTorch would, and no others."""
import ctypes

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


def test_an_error_of_an_earlier_call_is_not_this_calls():
    """Some other CUDA call of the program has failed on the host (a device that is not there)."""
    cudart = ctypes.CDLL("libcudart.so.12")
    x = torch.zeros(2, 1, 32, 32, device="cuda")
    at = torch.arange(2, dtype=torch.int32, device="cuda")
    cache, scales = torch.ones(2, 1, 32, 32, dtype=torch.int8, device="cuda"), torch.ones(2, 1, 32, device="cuda")
    torch.cuda.synchronize()
    assert cudart.cudaSetDevice(4096) != 0
    try:
        kda.kda_state_store(x, at, cache, scales)
        assert cudart.cudaPeekAtLastError() != 0                  # its caller's to read
    finally:
        cudart.cudaGetLastError()
    assert not cache.any() and not scales.any()
