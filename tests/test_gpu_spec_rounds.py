"""Speculative decoding as it is run: prefill, the state cache, tree decode, verification
and commit together, in a row without waiting, on several streams and in a graph.

Tolerances (relative L2): outputs and commits as in test_gpu_tree.py; a state that went
through several commits adds their errors (each relative to a state of like size).
"""
import numpy as np
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import inputs as kin
from linear_attention_08_b200 import kda
from parity import rel_l2

pytestmark = pytest.mark.gpu

TOL_TREE = {torch.float32: 64 * 2.0 ** -24, torch.bfloat16: 2.0 ** -8 + 8 * 2.0 ** -11}
ROWS = ("q", "k", "v", "g", "beta")


def cuda(d):
    return {x: y.cuda() for x, y in d.items()}


def tree(c, p, **kw):
    return kda.kda_decode_tree(*(c[x] for x in ROWS), c["init_state"], parents=p, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rounds_against_the_recurrence(dtype):
    """Two layers, four rounds: prompt, snapshot into the cache and back, then per round a
    tree in both layers, its verification, and both layers' commits; everything is queued
    without waiting.  The committed states are those of the accepted tokens one by one."""
    N, H, T, V, L, rounds = 3, 2, 11, 1000, 2, 4
    lengths = [70, 33, 128]
    cu = kin.cu_seqlens_of(lengths)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    layers, want = [], []
    for layer in range(L):
        d = kin.make_inputs((sum(lengths),), H, 128, 128, dtype, seed=100 + layer, num_states=N, state_std=0.1)
        c = cuda(d)
        _, fin, _ = kda.kda_prefill(*(c[x] for x in ROWS), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                    init_state=c["init_state"], chunk=64, cu_seqlens_host=cu)
        cache = torch.zeros(5, H, 128, 128, dtype=torch.int8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.zeros(5, H, 128, device="cuda")
        kda.kda_state_store(fin, slots, cache, scales)
        layers.append(kda.kda_state_load(cache, scales, slots))
    torch.cuda.synchronize()
    for S in layers:
        want.append(S.double().cpu().numpy())

    log = []
    for r in range(rounds):
        parents = ref.make_tree(N, T, ("bushy", "holes", "chain", "ragged")[r], seed=30 + r)
        target, draft, tokens, uniforms = ref.make_probs(N, T, V, torch.float32, seed=40 + r, parents=parents)
        p = None if parents is None else parents.cuda()
        tok = [ref.make_tokens(N, T, H, 128, 128, dtype, seed=50 + 10 * r + layer) for layer in range(L)]
        log.append((parents, target, draft, tokens, uniforms, tok, p, [cuda(x) for x in tok],
                    [x.cuda() for x in (target, draft, tokens, uniforms)]))
    results = []
    for parents, _, _, _, _, _, p, rows, (target, draft, tokens, uniforms) in log:
        outs = [kda.kda_decode_tree(*(c[x] for x in ROWS), layers[i], parents=p) for i, c in enumerate(rows)]
        node, length, out_tokens = kda.kda_verify_tree(target, tokens, uniforms, draft_probs=draft, parents=p)
        for i, c in enumerate(rows):
            kda.kda_tree_commit(*(c[x] for x in ROWS[1:]), layers[i], node, parents=p)
        results.append((outs, node, length, out_tokens, [S.clone() for S in layers]))
    torch.cuda.synchronize()

    for r, ((parents, target, draft, tokens, uniforms, tok, *_), (outs, node, length, out_tokens, states)) in \
            enumerate(zip(log, results)):
        for a, b in zip((node, length, out_tokens), ref.verify(target, draft, tokens, parents, uniforms)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        for i in range(L):
            d = dict(tok[i], init_state=torch.from_numpy(want[i]))
            o, _, alive = ref.tree(d, parents)
            want[i] = ref.commit(d, parents, node.cpu().numpy())
            assert rel_l2(outs[i], o) <= TOL_TREE[dtype] + 32 * T * r * 2.0 ** -24
            assert not outs[i][torch.from_numpy(~alive).cuda()].any()
            assert rel_l2(states[i], want[i]) <= 32 * T * (r + 1) * 2.0 ** -24


@pytest.mark.parametrize("dims", [(128, 128), (64, 64)])
def test_calls_in_a_row_wait_for_each_other(dims):
    """Each call reads what the one before it wrote, back to back many times over; the same
    calls with a wait between any two give the same bits."""
    N, T, H, V, rounds = 40, 9, 8, 3000, 12
    d = cuda(ref.make_tokens(N, T, H, *dims, torch.bfloat16, seed=11))
    parents = ref.make_tree(N, T, "bushy", seed=12)
    target, draft, tokens, uniforms = (x.cuda() for x in ref.make_probs(N, T, V, torch.bfloat16, seed=13, parents=parents))
    p = parents.cuda()
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()

    def run(wait):
        stop = torch.cuda.synchronize if wait else (lambda: None)
        state = d["init_state"].clone()
        cache = torch.zeros(N, H, *dims, dtype=torch.int8, device="cuda")
        scales = torch.zeros(N, H, dims[0], device="cuda")
        out = torch.zeros_like(d["v"])
        rows = dict(d)
        seen = []
        for r in range(rounds):
            kda.kda_decode_tree(*(rows[x] for x in ROWS), state, parents=p, out=out); stop()
            node, length, toks = kda.kda_verify_tree(target, tokens, (uniforms + 0.13 * r) % 1.0, draft_probs=draft, parents=p); stop()
            kda.kda_tree_commit(*(rows[x] for x in ROWS[1:]), state, node, parents=p); stop()
            kda.kda_state_store(state, slots, cache, scales); stop()
            kda.kda_state_load(cache, scales, slots, states=state); stop()
            rows["v"] = (0.5 * out + 0.5 * d["v"]).contiguous() if dims[0] == dims[1] else rows["v"]
            seen += [out.clone(), node, toks, state.clone()]
        torch.cuda.synchronize()
        return seen

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [5, 20, 33, 64])
def test_every_unit_of_a_large_batch(T):
    """More units than are resident: the order of the sequences changes no bit of any, and
    some are checked against the recurrence."""
    N, H = 60, 24
    d = ref.make_tokens(N, T, H, 128, 128, torch.bfloat16, seed=14)
    parents = ref.make_tree(N, T, "ragged", seed=15)
    c, p = cuda(d), parents.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tree(c, p, dev_status=status)
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(4)).cuda()
    other = tree({x: y[perm].contiguous() for x, y in c.items()}, p[perm].contiguous(), dev_status=status)
    torch.cuda.synchronize()
    assert torch.equal(out[perm], other) and status.item() == 0
    for n in (0, 31, 59):
        one = {x: y[n:n + 1] for x, y in d.items()}
        want, _, _ = ref.tree(one, parents[n:n + 1])
        if want.any():
            assert rel_l2(out[n:n + 1], want) <= TOL_TREE[torch.bfloat16]
        else:
            assert not out[n:n + 1].any()


def test_decay_out_of_range_in_32_places():
    d = ref.make_tokens(2, 27, 2, 128, 128, torch.bfloat16, seed=16)
    d["g"][0] = -5.0
    d["g"][1, 20:, 1] = -30.0
    for kind in ("chain", "bushy", "holes"):
        parents = ref.make_tree(2, 27, kind, seed=17)
        want, _, _ = ref.tree(d, parents)
        got = tree(cuda(d), None if parents is None else parents.cuda())
        assert rel_l2(got, want) <= TOL_TREE[torch.bfloat16]


@pytest.mark.parametrize("T", [6, 30, 60])
@pytest.mark.parametrize("bits", [0x7fffffff, 0x7fc00000, 0x7f800000])
def test_no_number_in_the_state_reaches_its_column(T, bits):
    """NaN or infinity in one element of the state: its value column of every token is no
    number, the other columns are as before."""
    d = cuda(ref.make_tokens(1, T, 2, 128, 128, torch.bfloat16, seed=18))
    p = ref.make_tree(1, T, "bushy", seed=19).cuda()
    clean = tree(d, p)
    d["init_state"] = d["init_state"].clone()
    d["init_state"].view(torch.int32)[0, 1, 77, 40] = bits
    got = tree(d, p)
    assert not torch.isfinite(got[0, :, 1, 40]).any()
    got[0, :, 1, 40] = clean[0, :, 1, 40]
    assert torch.equal(got, clean)


def test_streams_side_by_side():
    """Trees of several sizes, a multi-token decode (which also holds tensor memory) and
    verifications on four streams at once, against one after the other.  Every tensor that a
    call reads or writes lives until the end: the allocator knows of the current stream only."""
    jobs, none = [], torch.zeros(40, dtype=torch.int32, device="cuda")
    for i, (T, N, dims) in enumerate([(12, 30, (128, 128)), (30, 12, (128, 128)), (60, 8, (128, 128)), (16, 30, (64, 128))]):
        d = cuda(ref.make_tokens(N, T, 16, *dims, torch.bfloat16, seed=20 + i))
        p = ref.make_tree(N, T, "ragged", seed=24 + i).cuda()
        jobs.append(lambda s, d=d, p=p: tree(d, p, stream=s))
    m = cuda(ref.make_tokens(40, 8, 16, 128, 128, torch.bfloat16, seed=29))
    jobs.append(lambda s: kda.kda_decode_multi(*(m[x] for x in ROWS), m["init_state"], stream=s, accept_len=none))
    v = [x.cuda() for x in ref.make_probs(20, 6, 9000, torch.float32, seed=28)]
    jobs.append(lambda s: kda.kda_verify_tree(v[0], v[2], v[3], draft_probs=v[1], stream=s))
    same = lambda a, b: all(map(torch.equal, a, b)) if isinstance(a, tuple) else torch.equal(a, b)
    alone = [j(None) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for r in range(6):
        for i, j in enumerate(jobs):
            got.append((i, j(streams[(i + r) % 4])))
    torch.cuda.synchronize()
    for i, x in got:
        assert same(x, alone[i])


def test_outputs_belong_to_the_stream_they_are_made_on():
    """Outputs of a call on another stream, dropped at once: their memory is not given to
    the current stream's tensors while that stream still writes it."""
    d = cuda(ref.make_tokens(64, 16, 32, 128, 128, torch.bfloat16, seed=70))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        tree(d, None, stream=s)                       # 8 MB, dropped
        x = torch.full_like(d["v"], 3.0)
        s.synchronize()
        assert (x == 3).all()
    y = tree(d, None, stream=s)
    s.synchronize()
    assert torch.equal(y, tree(d, None))


def test_a_round_in_a_graph():
    """One round captured and replayed with other inputs, against the same calls eager."""
    N, T, H, V = 6, 10, 4, 2000
    d = cuda(ref.make_tokens(N, T, H, 128, 128, torch.bfloat16, seed=61))
    parents = ref.make_tree(N, T, "bushy", seed=62).cuda()
    target, draft, tokens, uniforms = (x.cuda() for x in ref.make_probs(N, T, V, torch.bfloat16, seed=63, parents=parents.cpu()))
    state, out = d["init_state"].clone(), torch.empty_like(d["v"])
    node, length = (torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(2))
    toks = torch.empty(N, T + 1, dtype=torch.int32, device="cuda")

    def go():
        kda.kda_decode_tree(*(d[x] for x in ROWS), state, parents=parents, out=out)
        kda.kda_verify_tree(target, tokens, uniforms, draft_probs=draft, parents=parents, accept_node=node,
                            accept_len=length, out_tokens=toks)
        kda.kda_tree_commit(*(d[x] for x in ROWS[1:]), state, node, parents=parents)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
        go()
    uniforms.copy_(torch.rand(N, T + 1, generator=torch.Generator().manual_seed(64)))
    parents.copy_(ref.make_tree(N, T, "random", seed=65))
    state.copy_(d["init_state"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (state, out, node, length, toks)]
    state.copy_(d["init_state"])
    for _ in range(4):
        go()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (state, out, node, length, toks)))


@pytest.mark.parametrize("dims", [(128, 128), (128, 32), (32, 64)])
def test_commit_of_a_large_batch_in_place(dims):
    """More items than are resident, accepted paths of zero to T tokens, in place and not."""
    N, T, H = 150, 21, 16
    d = cuda(ref.make_tokens(N, T, H, *dims, torch.bfloat16, seed=66))
    parents = ref.make_tree(N, T, "holes", seed=67)
    accept = torch.randint(-2, T + 2, (N,), generator=torch.Generator().manual_seed(68)).to(torch.int32)
    args = [d[x] for x in ROWS[1:]] + [d["init_state"], accept.cuda()]
    out = kda.kda_tree_commit(*args, parents=parents.cuda(), state_out=torch.empty_like(d["init_state"]))
    args[4] = d["init_state"].clone()
    assert torch.equal(kda.kda_tree_commit(*args, parents=parents.cuda()), out)
    some = slice(0, N, 29)
    sub = {x: y[some].cpu() for x, y in d.items()}
    assert rel_l2(out[some], ref.commit(sub, parents[some], accept[some].numpy())) <= 32 * T * 2.0 ** -24


def test_probabilities_below_the_normal_numbers():
    """FP32 numbers under 2^-126 count with their values: a token of 2^-140 is accepted at
    u = 0, and a row that holds nothing else is drawn from."""
    N, T, V = 4, 2, 40
    target, d, tokens, uniforms = ref.make_probs(N, T, V, torch.float32, seed=69)
    target[0, 0, tokens[0, 0].long()] = 2.0 ** -140
    uniforms[0, 0] = 0.0
    target[1] = 0
    target[1, :, 7], target[1, :, 9] = 2.0 ** -130, 3 * 2.0 ** -130
    uniforms[1, T] = 0.3
    d[2, :, 5] = 2.0 ** -149
    target[3] = -0.0
    for draft in (d, None):
        got = kda.kda_verify_tree(target.cuda(), tokens.cuda(), uniforms.cuda(),
                                  draft_probs=None if draft is None else draft.cuda())
        for a, b in zip(got, ref.verify(target, draft, tokens, None, uniforms)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
