"""Verification over clusters of every size, and numbers that are no probabilities."""
import numpy as np
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import kda
from test_gpu_verify import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("N", [3, 30, 60, 120, 160])
def test_every_cluster_size(dtype, draft, N):
    """8, 8, 4, 2 and 1 CTAs a sequence by the size of the batch (BF16 rows of 33001 elements, FP32 of
    17001, are long enough for all of them), with the drawn token in every CTA's slice."""
    T, V = 3, 33001 if dtype == torch.bfloat16 else 17001
    parents = ref.make_tree(N, T, "bushy", seed=101)
    target, d, tokens, uniforms = ref.make_probs(N, T, V, dtype, seed=102, parents=parents)
    uniforms[:, T] = (torch.arange(N) + 0.5) / N          # the border moves through the row
    uniforms[::7, T] = 1.0 - 2.0 ** -24
    uniforms[1::7, :T] = 1.0 - 2.0 ** -24                   # refusals
    check(target, d if draft else None, tokens, parents, uniforms)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), -0.5, -0.0])
def test_what_is_not_above_zero_counts_as_zero(dtype, bad):
    """At a drafted token itself, too: a draft that gives it no probability cannot refuse it."""
    N, T, V = 6, 4, 500
    parents = ref.make_tree(N, T, "bushy", seed=103)
    target, d, tokens, uniforms = ref.make_probs(N, T, V, dtype, seed=104, parents=parents)
    uniforms[:, :T] = 0.999
    for n in range(0, N, 2):
        for i in range(T):
            d[n, int(parents[n, i]) + 1 if parents[n, i] < T - 1 else 0, int(tokens[n, i])] = bad
    target[1, :, 3:9] = bad
    target[3, 0, int(tokens[3, 0])] = bad
    args = [x.cuda() for x in (target, tokens, uniforms)]
    got = kda.kda_verify_tree(*args, draft_probs=d.cuda(), parents=parents.cuda())
    zero = lambda x: torch.where(x > 0, x, torch.zeros_like(x))
    want = ref.verify(zero(target), zero(d), tokens, parents, uniforms)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
