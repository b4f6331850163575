"""kda_verify_tree against the definition in 64 bits: whole numbers, compared exactly."""
import numpy as np
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import kda

pytestmark = pytest.mark.gpu


def check(target, draft, tokens, parents, uniforms):
    cu = lambda x: None if x is None else x.cuda()
    got = kda.kda_verify_tree(cu(target), cu(tokens), cu(uniforms), draft_probs=cu(draft), parents=cu(parents))
    torch.cuda.synchronize()
    want = ref.verify(target, draft, tokens, parents, uniforms)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("T,kind", [(1, "chain"), (5, "chain"), (8, "bushy"), (13, "star"), (24, "ragged"), (33, "holes"), (64, "random")])
@pytest.mark.parametrize("V", [1, 2, 37, 1000, 4096])
def test_verify_against_definition(dtype, draft, T, kind, V):
    N = 6
    parents = ref.make_tree(N, T, kind, seed=T)
    target, d, tokens, uniforms = ref.make_probs(N, T, V, dtype, seed=61 + T, parents=parents)
    check(target, d if draft else None, tokens, parents, uniforms)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50257, 65536, 131071])
def test_verify_large_vocabulary(dtype, V):
    N, T = 4, 5
    parents = ref.make_tree(N, T, "bushy", seed=4)
    check(*(lambda t, d, k, u: (t, d, k, parents, u))(*ref.make_probs(N, T, V, dtype, seed=62, parents=parents)))


@pytest.mark.parametrize("N", [1, 3, 80, 200, 600])
def test_verify_batch_sizes(N):
    """Every cluster size, one to eight CTAs a sequence."""
    T, V = 4, 777
    target, d, tokens, uniforms = ref.make_probs(N, T, V, torch.float32, seed=63)
    node, length, _ = check(target, d, tokens, None, uniforms)
    assert (length == node + 1).all()
    if N >= 80:
        assert set(length.tolist()) == set(range(T + 1))


def test_random_numbers_at_the_ends():
    """0 draws the first token with a probability; the largest FP32 below 1, and 1 itself
    (outside the documented range), the last one at most."""
    V, T = 300, 2
    for last in (0.0, 1.0 - 2.0 ** -24, 1.0):
        target, d, tokens, uniforms = ref.make_probs(3, T, V, torch.float32, seed=64)
        target[:, :, :7] = 0
        target[:, :, -9:] = 0
        target /= target.sum(-1, keepdim=True)
        uniforms[:, T] = last
        check(target, d, tokens, None, uniforms)
        uniforms[:, :T] = 1.0 - 2.0 ** -24
        check(target, d, tokens, None, uniforms)
        check(target, None, tokens, None, uniforms)


def test_certain_rows_zero_rows_and_equal_rows():
    N, T, V = 4, 3, 64
    target, d, tokens, uniforms = ref.make_probs(N, T, V, torch.float32, seed=65)
    target[0] = 0
    target[0, :, 5] = 1.0                     # one token has everything
    tokens[0] = torch.tensor([5, 6, 5])
    target[1, :T] = d[1]                      # target = draft: always accepted
    target[2] = 0                             # no probability at all
    target[3, 0] = d[3, 0] * 0.5              # below the draft everywhere: nothing is left
    d[3, 0, tokens[3, 0].long()] *= 4
    uniforms[3, 0] = 0.9
    for draft in (d, None):
        check(target, draft, tokens, None, uniforms)
    got = kda.kda_verify_tree(target.cuda(), tokens.cuda(), uniforms.cuda(), draft_probs=d.cuda())
    assert got[1][1] == T and got[2][2, 0] == -1 and got[2][0].tolist() == [5, 5, -1, -1]


def test_tokens_outside_the_vocabulary():
    N, T, V = 3, 4, 100
    target, d, tokens, uniforms = ref.make_probs(N, T, V, torch.bfloat16, seed=66)
    tokens[0, 0], tokens[1, 1], tokens[2, 2] = -1, V, 2 ** 31 - 1
    for draft in (d, None):
        check(target, draft, tokens, None, uniforms)


@pytest.mark.parametrize("draft", [True, False])
def test_repeated_siblings(draft):
    """The same token proposed several times after one context."""
    N, T, V = 5, 6, 50
    target, d, tokens, uniforms = ref.make_probs(N, T, V, torch.float32, seed=67)
    tokens[:] = tokens[:, :1]
    parents = torch.full((N, T), -1, dtype=torch.int32)
    check(target, d if draft else None, tokens, parents, uniforms)


def test_unaligned_rows_and_outputs_in_larger_buffers():
    N, T, V = 3, 4, 4001
    target, d, tokens, uniforms = ref.make_probs(N, T, V, torch.bfloat16, seed=68)
    big = torch.zeros(target.numel() + 3, dtype=torch.bfloat16, device="cuda")
    t = big[3:].view(target.shape)
    t.copy_(target)
    outs = torch.full((64,), -77, dtype=torch.int32, device="cuda")
    node, length, out = outs[1:4], outs[7:10], outs[13:13 + N * (T + 1)].view(N, T + 1)
    kda.kda_verify_tree(t, tokens.cuda(), uniforms.cuda(), draft_probs=d.cuda(), accept_node=node,
                        accept_len=length, out_tokens=out)
    want = ref.verify(target, d, tokens, None, uniforms)
    for a, b in zip((node, length, out), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    rest = outs.cpu().numpy()
    assert (rest[[0, 4, 5, 6, 10, 11, 12]] == -77).all() and (rest[13 + N * (T + 1):] == -77).all()


def test_draws_follow_the_target():
    """Accepted and drawn first tokens together have the target's frequencies: chi-square
    over 8 tokens (7 degrees of freedom) below 24.3 (1 in 1000), with a fixed seed."""
    N, T, V = 40000, 3, 8
    gen = torch.Generator().manual_seed(70)
    p = torch.softmax(torch.randn(V, generator=gen), 0)
    q = torch.softmax(torch.randn(V, generator=gen), 0)
    target = p.expand(N, T + 1, V).contiguous().cuda()
    draft = q.expand(N, T, V).contiguous().cuda()
    tokens = torch.multinomial(q.expand(N, V), T, replacement=True, generator=gen).to(torch.int32)
    parents = torch.tensor([-1, -1, 0], dtype=torch.int32).expand(N, T).contiguous()
    uniforms = torch.rand(N, T + 1, generator=gen)
    for dr in (draft, None):
        tok = tokens if dr is not None else torch.tensor([1, 4, 2], dtype=torch.int32).expand(N, T).contiguous()
        _, _, out = kda.kda_verify_tree(target, tok.cuda(), uniforms.cuda(), draft_probs=dr, parents=parents.cuda())
        seen = torch.bincount(out[:, 0].cpu().long(), minlength=V).double()
        chi = float(((seen - N * p.double()) ** 2 / (N * p.double())).sum())
        assert chi < 24.3


def test_verify_graph_and_two_streams():
    N, T, V = 16, 4, 5000
    target, d, tokens, uniforms = (x.cuda() for x in ref.make_probs(N, T, V, torch.float32, seed=71))
    outs = [torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(2)] + [
        torch.empty(N, T + 1, dtype=torch.int32, device="cuda")]
    go = lambda: kda.kda_verify_tree(target, tokens, uniforms, draft_probs=d, accept_node=outs[0],
                                     accept_len=outs[1], out_tokens=outs[2])
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    uniforms.copy_(torch.rand(N, T + 1, generator=torch.Generator().manual_seed(72)))
    graph.replay()
    torch.cuda.synchronize()
    want = ref.verify(target, d, tokens.cpu(), None, uniforms)
    for a, b in zip(outs, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    pair = [kda.kda_verify_tree(target, tokens, uniforms, draft_probs=d, stream=s)
            for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*pair))
