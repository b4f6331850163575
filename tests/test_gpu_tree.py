"""kda_decode_tree and kda_tree_commit against the recurrence in 64 bits.

Tolerances (relative L2).  FP32 inputs: exp to 2 ulp in each of two factors (4
half-steps each), operands split in two TF32 terms (what is dropped: 2^-22 of a
product, twice), FP32 accumulation over 16 tiles: 16 + 8 + 32 half-steps of 2^-24,
taken as 64.  BF16 inputs: the rounding of out (2^-8) and eight TF32 operand
roundings (2^-11 each) along S0 -> Vn -> out.  Commit: FP32 in both cases, up to 32
half-steps a token (exp 4, the gate 1, a sum of 128 terms in 16 + 3 steps, the
correction and the update 4).
"""
import numpy as np
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import kda
from parity import rel_l2

pytestmark = pytest.mark.gpu

TOL_TREE = {torch.float32: 64 * 2.0 ** -24, torch.bfloat16: 2.0 ** -8 + 8 * 2.0 ** -11}


def cuda(d):
    return {x: y.cuda() for x, y in d.items()}


def run_tree(d, parents, **kw):
    c = cuda(d)
    return kda.kda_decode_tree(c["q"], c["k"], c["v"], c["g"], c["beta"], c["init_state"],
                               parents=None if parents is None else parents.cuda(), **kw)


def run_commit(d, parents, accept, **kw):
    c = cuda(d)
    return kda.kda_tree_commit(c["k"], c["v"], c["g"], c["beta"], c["init_state"],
                               torch.as_tensor(accept, dtype=torch.int32).cuda(),
                               parents=None if parents is None else parents.cuda(), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dims", [(32, 32), (32, 128), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("T,kind", [(1, "chain"), (7, "bushy"), (8, "star"), (9, "chain"), (16, "random"),
                                    (17, "holes"), (33, "ragged"), (64, "random")])
def test_tree_against_recurrence(dtype, dims, T, kind):
    N, H = 3, 2
    d = ref.make_tokens(N, T, H, *dims, dtype, seed=41 + T)
    parents = ref.make_tree(N, T, kind, seed=T)
    out = run_tree(d, parents)
    torch.cuda.synchronize()
    want, _, alive = ref.tree(d, parents)
    assert rel_l2(out, want) <= TOL_TREE[dtype]
    assert not out[torch.from_numpy(~alive).cuda()].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [16, 40, 64])
def test_tree_deep_decay(dtype, T):
    """Chains whose cumulative log-decay passes -80, and single resets to nothing: the
    factored products would overflow, so L and P are formed pair by pair."""
    N, H = 2, 2
    d = ref.make_tokens(N, T, H, 128, 128, dtype, seed=7)
    d["g"][0] = -5.0
    d["g"][1, 3, 0, 5] = -1.0e4
    d["g"][1, :, 1, 77] = -40.0
    for kind in ("chain", "bushy"):
        parents = ref.make_tree(N, T, kind, seed=3)
        out = run_tree(d, parents)
        want, _, _ = ref.tree(d, parents)
        assert rel_l2(out, want) <= TOL_TREE[dtype]


def test_tree_large_keys():
    """Keys of size 10^3 push the factors past their limit before the decay does."""
    d = ref.make_tokens(1, 12, 1, 64, 64, torch.float32, seed=8)
    d["k"] = d["k"] * 1.0e3
    d["beta"] = d["beta"] * 1.0e-6
    d["g"] = torch.full_like(d["g"], -5.0)
    parents = ref.make_tree(1, 12, "bushy", seed=2)
    want, _, _ = ref.tree(d, parents)
    assert rel_l2(run_tree(d, parents), want) <= TOL_TREE[torch.float32]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_empty_places_reach_nothing(dtype):
    """NaN and infinity in every input of the empty places change no bit elsewhere."""
    N, T, H = 3, 20, 2
    d = ref.make_tokens(N, T, H, 128, 128, dtype, seed=9)
    parents = ref.make_tree(N, T, "holes", seed=5)
    _, _, alive = ref.tree(d, parents)
    clean = run_tree(d, parents)
    dead = torch.from_numpy(~alive)
    for x, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("g", float("-inf")), ("beta", float("nan"))):
        d[x] = d[x].clone()
        d[x][dead] = bad
    assert torch.equal(run_tree(d, parents), clean)


def test_tree_chain_equals_explicit_chain_and_decode_multi():
    N, T, H = 4, 8, 3
    d = ref.make_tokens(N, T, H, 128, 128, torch.float32, seed=10)
    chain = (torch.arange(T, dtype=torch.int32) - 1).expand(N, T).contiguous()
    a, b = run_tree(d, None), run_tree(d, chain)
    assert torch.equal(a, b)
    c = cuda(d)
    m = kda.kda_decode_multi(c["q"], c["k"], c["v"], c["g"], c["beta"], c["init_state"].clone())
    assert rel_l2(a, m.double().cpu().numpy()) <= 1e-5


def test_tree_reads_the_state_only_and_fills_out():
    d = cuda(ref.make_tokens(2, 5, 2, 128, 128, torch.bfloat16, seed=11))
    keep = d["init_state"].clone()
    buf = torch.full((2 * 5 * 2 * 128 + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[256:256 + 2 * 5 * 2 * 128].view(2, 5, 2, 128)
    kda.kda_decode_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], d["init_state"], out=out)
    assert torch.equal(keep, d["init_state"])
    assert (buf[:256] == 7).all() and (buf[-256:] == 7).all()


def test_tree_many_units_and_streams():
    """More units than fit at once, on two streams at a time; every unit checked against a
    second run and some against the recurrence."""
    N, T, H = 96, 12, 32
    d = ref.make_tokens(N, T, H, 128, 128, torch.bfloat16, seed=12)
    parents = ref.make_tree(N, T, "ragged", seed=6)
    c, p = cuda(d), parents.cuda()
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        outs.append(kda.kda_decode_tree(c["q"], c["k"], c["v"], c["g"], c["beta"], c["init_state"],
                                        parents=p, stream=s))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    for n in (0, 41, 95):
        one = {x: y[n:n + 1] for x, y in d.items()}
        want, _, _ = ref.tree(one, parents[n:n + 1])
        assert rel_l2(outs[0][n:n + 1], want) <= TOL_TREE[torch.bfloat16]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dims", [(32, 32), (32, 64), (64, 128), (128, 32), (128, 128)])
@pytest.mark.parametrize("T,kind", [(1, "chain"), (8, "bushy"), (23, "holes"), (64, "chain")])
def test_commit_against_recurrence(dtype, dims, T, kind):
    N, H = 7, 2
    d = ref.make_tokens(N, T, H, *dims, dtype, seed=51 + T)
    parents = ref.make_tree(N, T, kind, seed=T + 1)
    accept = np.array([-1, 0, T - 1, T // 2, T, -2 ** 31, 2 ** 31 - 1])
    want = ref.commit(d, parents, accept)
    out = torch.full((N, H, *dims), float("nan"), device="cuda")
    kept = run_commit(d, parents, accept, state_out=out)
    assert kept is out
    inplace = run_commit(d, parents, accept)
    torch.cuda.synchronize()
    assert torch.equal(out, inplace)
    assert rel_l2(out, want) <= 32 * T * 2.0 ** -24
    for n in (0, 4, 5, 6):                       # nothing accepted: the same bits
        assert torch.equal(out[n].cpu(), d["init_state"][n])


def test_commit_extreme_decay():
    d = ref.make_tokens(2, 16, 2, 128, 128, torch.bfloat16, seed=52)
    d["g"][0, :, 0, 5] = -1.0e4
    d["g"][1] = -5.0
    accept = np.array([15, 15])
    got = run_commit(d, None, accept)
    assert torch.isfinite(got).all()
    assert rel_l2(got, ref.commit(d, None, accept)) <= 32 * 16 * 2.0 ** -24


def test_commit_continues_the_tree():
    """The state of an accepted token gives its successors the outputs they had in the tree."""
    N, H = 3, 2
    d = ref.make_tokens(N, 9, H, 128, 128, torch.float32, seed=53)
    parents = torch.tensor([[-1, 0, 1, 1, 3, 3, 5, -1, 7]] * N, dtype=torch.int32)
    c = cuda(d)
    out = run_tree(d, parents)
    state = kda.kda_tree_commit(c["k"], c["v"], c["g"], c["beta"], c["init_state"],
                                torch.full((N,), 3, dtype=torch.int32, device="cuda"), parents=parents.cuda())
    rest = torch.tensor([[-1, -1, 1]] * N, dtype=torch.int32).cuda()
    sub = {x: c[x][:, 4:7].contiguous() for x in ("q", "k", "v", "g", "beta")}
    again = kda.kda_decode_tree(sub["q"], sub["k"], sub["v"], sub["g"], sub["beta"], state, parents=rest)
    assert rel_l2(again, out[:, 4:7].double().cpu().numpy()) <= 2 * TOL_TREE[torch.float32] + 64 * 2.0 ** -24


def test_graph_capture_tree_and_commit():
    d = cuda(ref.make_tokens(4, 6, 2, 128, 128, torch.bfloat16, seed=54))
    parents = ref.make_tree(4, 6, "bushy", seed=9).cuda()
    accept = torch.tensor([0, 5, -1, 3], dtype=torch.int32, device="cuda")
    out, after = torch.empty_like(d["v"]), torch.empty_like(d["init_state"])

    def go():
        kda.kda_decode_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], d["init_state"], parents=parents, out=out)
        kda.kda_tree_commit(d["k"], d["v"], d["g"], d["beta"], d["init_state"], accept, parents=parents, state_out=after)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    d["v"].mul_(2)
    accept.copy_(torch.tensor([5, 0, 2, -1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone(), after.clone()
    go()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], after)
