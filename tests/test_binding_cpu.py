"""The native part of the binding without a GPU: what it refuses, and with which error."""
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import kda


def tokens():
    d = ref.make_tokens(2, 3, 2, 32, 32, torch.float32, seed=1)
    return [d[x] for x in ("q", "k", "v", "g", "beta", "init_state")]


def test_host_tensors_are_refused_everywhere():
    a = tokens()
    node = torch.zeros(2, dtype=torch.int32)
    t, dr, tok, u = ref.make_probs(2, 3, 9, torch.float32, seed=2)
    x, at = torch.zeros(2, 1, 32, 32), torch.zeros(2, dtype=torch.int32)
    cache, scales = torch.zeros(4, 1, 32, 32, dtype=torch.int8), torch.zeros(4, 1, 32)
    for call in (lambda: kda.kda_decode_tree(*a), lambda: kda.kda_tree_commit(*a[1:], node),
                 lambda: kda.kda_verify_tree(t, tok, u, draft_probs=dr),
                 lambda: kda.kda_state_store(x, at, cache, scales), lambda: kda.kda_state_load(cache, scales, at)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_types_shapes_and_arguments_that_are_no_tensors():
    a = tokens()
    for bad in (None, [1.0], "k"):
        with pytest.raises(TypeError, match="k must be a tensor"):
            kda.kda_decode_tree(a[0], bad, *a[2:])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        kda.kda_decode_tree(*[x.half() for x in a[:3]], *a[3:])
    with pytest.raises(ValueError, match="dimensions"):
        kda.kda_decode_tree(a[0], a[1][0], *a[2:])
    t, dr, tok, u = ref.make_probs(2, 3, 9, torch.float32, seed=2)
    with pytest.raises(TypeError):
        kda.kda_verify_tree(t.double(), tok, u)
    with pytest.raises(ValueError, match="prefix"):
        kda.kda_verify_tree(t[:, :1].contiguous(), tok, u)
    with pytest.raises(ValueError, match="dimensions"):
        kda.kda_state_load(torch.zeros(4, 32, 32, dtype=torch.int8), torch.zeros(4, 32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError, match="float8_e4m3fn or int8"):
        kda.kda_state_load(torch.zeros(4, 1, 32, 32), torch.zeros(4, 1, 32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(AttributeError):
        kda.kda_decode_tree(*a, stream=7)


def test_wrong_numbers_of_arguments():
    native = kda._native()
    for f in (native.decode_tree, native.tree_commit, native.verify_tree, native.state_store, native.state_load):
        with pytest.raises(TypeError, match="arguments"):
            f(1, 2)
