"""Speculative decoding and the state cache without a GPU: refusals of the C ABI and of
the binding before any launch, and the tests' 64-bit references against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import spec_ref as ref
from linear_attention_08_b200 import kda

BAD, UNSUP = kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED


def P(x):
    return None if x is None else ctypes.c_void_p(x)


A, B, C, D, E, F, G, I = ((1 << 30) * (4 * i + 4) for i in range(8))   # far apart, never dereferenced


def tree_call(fn, swap=None, shape=None, T=4):
    names = {"kda_decode_tree": ["q", "k", "v", "g", "beta", "state", "parents", "out"],
             "kda_tree_commit": ["k", "v", "g", "beta", "state", "state_out", "parents", "accept_node"]}[fn]
    args = dict(zip(names, (A, B, C, D, E, F, G, I)))
    args.update(swap or {})
    s = shape or kda.make_shape(3, 12, 2, 64, 64, 0, 1)
    return getattr(kda.load(), fn)(*(P(args[x]) for x in names), T, ctypes.byref(s), None)


@pytest.mark.parametrize("fn", ["kda_decode_tree", "kda_tree_commit"])
def test_tree_calls_refuse_bad_arguments(fn):
    mk = kda.make_shape
    for T in (0, -1, 65, 5):                                   # 5: total_tokens != N * T
        assert tree_call(fn, T=T) == BAD
    assert tree_call(fn, shape=mk(3, 12, 2, 48, 64, 0, 1)) == UNSUP
    assert tree_call(fn, shape=mk(3, 12, 2, 64, 256, 0, 1)) == UNSUP
    assert tree_call(fn, shape=mk(0, 0, 2, 64, 64, 0, 1)) == BAD
    assert tree_call(fn, shape=mk(3, 12, 0, 64, 64, 0, 1)) == BAD
    assert tree_call(fn, shape=mk(3, 12, 2, 64, 64, 0, 2)) == BAD
    for x in ("k", "v", "g", "state"):
        assert tree_call(fn, {x: None}) == BAD
        assert tree_call(fn, {x: A + 8}) == BAD
    for x in ("beta", "parents"):
        assert tree_call(fn, {x: A + 2}) == BAD
    assert tree_call(fn, {"beta": None}) == BAD


def test_tree_calls_refuse_overlaps():
    state = 3 * 2 * 64 * 64 * 4
    rows = 12 * 2 * 64 * 2
    for x, n in (("q", rows), ("k", rows), ("v", rows), ("g", 2 * rows), ("beta", 96), ("state", state), ("parents", 48)):
        base = dict(zip(["q", "k", "v", "g", "beta", "state", "parents"], (A, B, C, D, E, F, G)))[x]
        assert tree_call("kda_decode_tree", {"out": base}) == BAD
        assert tree_call("kda_decode_tree", {"out": base + n - 16}) == BAD
    assert tree_call("kda_tree_commit", {"state_out": E + state - 16}) == BAD      # state is E here
    assert tree_call("kda_tree_commit", {"state_out": E - 16}) == BAD
    for x, at in (("k", A), ("v", B), ("g", C), ("beta", D), ("parents", G), ("accept_node", I)):
        assert tree_call("kda_tree_commit", {"state_out": at}) == BAD
    assert tree_call("kda_tree_commit", {"accept_node": None}) == BAD
    assert tree_call("kda_tree_commit", {"accept_node": I + 1}) == BAD


def verify_call(swap=None, N=3, T=4, V=100, dtype=0):
    names = ["target", "draft", "tokens", "parents", "uniforms", "node", "length", "out"]
    args = dict(zip(names, (A, B, C, D, E, F, G, I)))
    args.update(swap or {})
    return kda.load().kda_verify_tree(*(P(args[x]) for x in names), N, T, V, dtype, None)


def test_verify_refuses_bad_arguments():
    for kw in (dict(N=0), dict(N=-1), dict(T=0), dict(T=65), dict(V=0), dict(V=-5), dict(dtype=2), dict(dtype=-1)):
        assert verify_call(**kw) == BAD
    assert verify_call(V=(1 << 30) + 1) == UNSUP
    assert verify_call(N=(1 << 27) + 1) == UNSUP
    for x in ("target", "tokens", "uniforms", "node", "length", "out"):
        assert verify_call({x: None}) == BAD
    for x in ("target", "draft", "tokens", "parents", "uniforms", "node", "length", "out"):
        assert verify_call({x: A + (4 << 30) * 9 + 2}) == BAD          # FP32 and int32: 4-byte aligned
    assert verify_call({"target": A + 1}, dtype=1) == BAD
    for x in ("node", "length", "out"):
        for at in (A, B, C, D, E, A + 3 * 5 * 100 * 4 - 4):
            assert verify_call({x: at}) == BAD
    assert verify_call({"node": I}) == BAD and verify_call({"length": F + 8}) == BAD


def cache_call(fn, swap=None, shape=None, slots=7, dtype=0):
    args = dict(states=A, where=B, cache=C, scales=D)
    args.update(swap or {})
    s = shape or kda.make_shape(3, 3, 2, 64, 64, 0, 0)
    order = ["states", "where", "cache", "scales"] if fn == "kda_state_store" else ["cache", "scales", "where", "states"]
    return getattr(kda.load(), fn)(*(P(args[x]) for x in order), slots, dtype, ctypes.byref(s), None)


@pytest.mark.parametrize("fn", ["kda_state_store", "kda_state_load"])
def test_cache_calls_refuse_bad_arguments(fn):
    assert cache_call(fn, slots=0) == BAD and cache_call(fn, slots=-3) == BAD
    assert cache_call(fn, slots=1 << 31) == UNSUP
    assert cache_call(fn, dtype=2) == BAD and cache_call(fn, dtype=-1) == BAD
    assert cache_call(fn, shape=kda.make_shape(3, 3, 2, 16, 64, 0, 0)) == UNSUP
    assert cache_call(fn, shape=kda.make_shape(0, 0, 2, 64, 64, 0, 0)) == BAD
    for x in ("states", "cache", "scales"):
        assert cache_call(fn, {x: None}) == BAD
        assert cache_call(fn, {x: A + (4 << 30) * 9 + 4}) == BAD
    assert cache_call(fn, {"where": None}) == BAD and cache_call(fn, {"where": B + 2}) == BAD
    n_cache, n_scale = 7 * 2 * 64 * 64, 7 * 2 * 64 * 4
    assert cache_call(fn, {"states": C + n_cache - 16}) == BAD
    assert cache_call(fn, {"states": D + n_scale - 16}) == BAD
    assert cache_call(fn, {"scales": C}) == BAD
    assert cache_call(fn, {"where": A + 16}) == BAD and cache_call(fn, {"where": C}) == BAD


def test_null_shape_is_refused():
    lib = kda.load()
    p = P(A)
    assert lib.kda_decode_tree(p, p, p, p, p, p, p, P(I), 4, None, None) == BAD
    assert lib.kda_tree_commit(p, p, p, p, p, P(I), p, p, 4, None, None) == BAD
    assert lib.kda_state_store(p, P(B), P(C), P(D), 4, 0, None, None) == BAD
    assert lib.kda_state_load(p, P(B), P(C), P(D), 4, 0, None, None) == BAD


def test_binding_checks_tensors():
    d = ref.make_tokens(2, 3, 2, 32, 32, torch.float32, seed=1)
    args = [d[x] for x in ("q", "k", "v", "g", "beta", "init_state")]
    with pytest.raises(ValueError):                            # host tensors
        kda.kda_decode_tree(*args)
    for i, bad in ((0, args[0].double()), (3, args[3].bfloat16()), (5, args[5].half())):
        with pytest.raises((TypeError, ValueError)):
            kda.kda_decode_tree(*(args[:i] + [bad] + args[i + 1:]))
    with pytest.raises(ValueError):
        kda.kda_tree_commit(*args[1:], torch.zeros(2, dtype=torch.int32))
    t, dr, tok, u = ref.make_probs(2, 3, 9, torch.float32, seed=2)
    with pytest.raises((TypeError, ValueError)):
        kda.kda_verify_tree(t, tok.long(), u, draft_probs=dr)
    with pytest.raises(TypeError):
        kda.kda_verify_tree(t.half(), tok, u)
    x = torch.zeros(2, 1, 32, 32)
    with pytest.raises(TypeError):
        kda.kda_state_store(x, torch.zeros(2, dtype=torch.int32), torch.zeros(4, 1, 32, 32), torch.zeros(4, 1, 32))


# ---- the references themselves

def test_tree_reference_against_the_oracle():
    """Every root-to-token path of a tree is a sequence of its own."""
    N, T, H = 2, 7, 2
    d = ref.make_tokens(N, T, H, 32, 64, torch.float32, seed=3)
    parents = ref.make_tree(N, T, "random", seed=4)
    out, states, alive = ref.tree(d, parents)
    assert alive.all()
    for n in range(N):
        for t in range(T):
            path = ref.path_to(parents[n], t, T)
            seq = [d[x][n, path] for x in ("q", "k", "v", "g", "beta")]
            o, fin, _ = oracle.prefill(*seq, [0, len(path)], d["init_state"][n:n + 1])
            np.testing.assert_allclose(out[n, t], o[-1], rtol=1e-10, atol=1e-12)
            np.testing.assert_allclose(states[n, t], fin[0], rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(ref.commit(d, parents, [T - 1, -1])[1], d["init_state"][1].double())


@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_reference_keeps_the_target_distribution(with_draft):
    """The first token out, with the two drafted tokens and the random numbers summed
    over a fine grid, has the target's probabilities."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    M = 40
    grid = (np.arange(M) + 0.5) / M
    seen = np.zeros(3)
    u = np.array(np.meshgrid(grid, grid, grid, indexing="ij")).reshape(3, -1).T[::7]
    pairs = [(a, b, q[a] * q[b]) for a in range(3) for b in range(3)] if with_draft else [(2, 0, 1.0)]
    for a, b, w in pairs:
        n = len(u)
        _, _, out = ref.verify(np.broadcast_to(p, (n, 3, 3)), np.broadcast_to(q, (n, 2, 3)) if with_draft else None,
                               np.tile([a, b], (n, 1)), np.full((n, 2), -1), u)
        seen += w * np.bincount(out[:, 0], minlength=3) / n
    np.testing.assert_allclose(seen, p, atol=0.02)


def test_e4m3_reference_against_torch():
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(3, 2, 32, 64, generator=gen) * torch.exp(3 * torch.randn(3, 2, 32, 1, generator=gen))
    codes, scale = ref.quantise(x.numpy(), "e4m3")
    y = (x / torch.from_numpy(scale)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(codes, y.double().numpy())
