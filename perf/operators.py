"""The operators of speculative decoding and of the state cache, as they are measured.

Five operators that belong together in a serving loop over recurrent KDA states:

* ``tree``   -- outputs of a tree of drafted tokens over each sequence's state;
* ``verify`` -- acceptance of drafted tokens against the target's probabilities
  from given random numbers, with the next token drawn from what is left;
* ``commit`` -- the state moved along the accepted path of the tree;
* ``store``  -- states quantised into the 8-bit state cache;
* ``load``   -- states read back from it.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, by the library's calls.  ``exact`` gives the same in 64 bits, token by
token, from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CACHES = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user's draft of eight tokens in a small tree: latency of one layer
        dict(name="tree_n1_t8", op="tree", n=1, t=8, h=32, dk=128, dv=128, dtype="bf16", kind="bushy", ragged=False),
        # the decode workload's batch (512 sequences, 32 heads), 16 drafted tokens each
        dict(name="tree_n512_t16", op="tree", n=512, t=16, h=32, dk=128, dv=128, dtype="bf16", kind="bushy", ragged=False),
        # big trees of uneven sizes over a small batch
        dict(name="tree_n43_t61_ragged", op="tree", n=43, t=61, h=32, dk=128, dv=128, dtype="bf16", kind="random", ragged=True),
        # the accepted path of the decode workload's batch, a few tokens each
        dict(name="commit_n512_t16", op="commit", n=512, t=16, h=32, dk=128, dv=128, dtype="bf16", kind="bushy", ragged=False),
        # FP32 with narrow keys, an odd batch, long chains
        dict(name="commit_n37_t23_f32", op="commit", n=37, t=23, h=5, dk=64, dv=128, dtype="f32", kind="chain", ragged=True),
        # one user's chain of five drafted tokens: latency
        dict(name="verify_n1_t5", op="verify", n=1, t=5, vocab=32000, dtype="f32", kind="chain", ragged=False, draft=True),
        # a served batch with a large vocabulary, chains of seven
        dict(name="verify_n64_t7", op="verify", n=64, t=7, vocab=131072, dtype="bf16", kind="chain", ragged=False, draft=True),
        # trees of drafted tokens, siblings drawn from one draft distribution, odd vocabulary
        dict(name="verify_n48_t24_tree", op="verify", n=48, t=24, vocab=50257, dtype="f32", kind="bushy", ragged=True, draft=True),
        # snapshots of a long prefill (one every 32K tokens of 1M) into the cache
        dict(name="store_n32_e4m3", op="store", n=32, slots=48, h=32, dk=128, dv=128, cache="e4m3"),
        # the prompt boundaries of a full batch into the cache
        dict(name="store_n512_int8", op="store", n=512, slots=520, h=32, dk=128, dv=128, cache="int8"),
        # a full batch resumed from cached prefixes, new sequences among them
        dict(name="load_n512_e4m3", op="load", n=512, slots=520, h=32, dk=128, dv=128, cache="e4m3"),
        # one resumed sequence: latency
        dict(name="load_n1_int8", op="load", n=1, slots=16, h=32, dk=128, dv=128, cache="int8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tree", "commit", "verify", "store", "load"])
    if op == "verify":
        t, vocab = _log(rng, 1, 64), _log(rng, 1000, 131072)
        n = _log(rng, 1, max(1, min(256, 64 * 8 * 131072 // ((t + 1) * vocab))))
        return dict(op=op, n=n, t=t, vocab=vocab, dtype=rng.choice(["f32", "bf16"]),
                    kind=rng.choice(["chain", "bushy", "random"]), ragged=rng.random() < 0.5, draft=rng.random() < 0.75)
    h, dk, dv = _log(rng, 1, 32), rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128])
    if op in ("tree", "commit"):
        t = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, min(512, 512 * 32 * 16 // (h * max(t, 16)))))
        return dict(op=op, n=n, t=t, h=h, dk=dk, dv=dv, dtype=rng.choice(["f32", "bf16", "bf16"]),
                    kind=rng.choice(["chain", "bushy", "random"]), ragged=rng.random() < 0.5)
    n = _log(rng, 1, min(512, 512 * 32 // h))
    return dict(op=op, n=n, slots=n + _log(rng, 1, 32), h=h, dk=dk, dv=dv, cache=rng.choice(["e4m3", "int8"]))


def work(case):
    c = case
    n = c["n"]
    if c["op"] == "verify":
        # per sequence: the last context's target row, its draft row, the drawn tokens' probabilities
        es = 2 if c["dtype"] == "bf16" else 4
        rows = 2 if c["draft"] else 1
        return {"bytes": n * (rows * c["vocab"] * es + c["t"] * (12 + 2 * es) + 4 * (c["t"] + 4)),
                "flops": n * 4 * c["vocab"]}
    h, dk, dv = c["h"], c["dk"], c["dv"]
    state = 4 * n * h * dk * dv
    if c["op"] in ("tree", "commit"):
        es, t = (2 if c["dtype"] == "bf16" else 4), c["t"]
        if c["op"] == "tree":
            rows = n * t * h * (2 * dk * es + 2 * dv * es + 4 * dk + 4)
            return {"bytes": state + rows + 4 * n * t, "flops": n * h * t * 4 * dk * dv}
        a = _mean_accepted(t)   # tokens on the accepted path
        rows = int(n * a * h * (dk * es + dv * es + 4 * dk + 4))
        return {"bytes": 2 * state + rows + 4 * n * (t + 1), "flops": int(n * h * a * 6 * dk * dv)}
    return {"bytes": state + state // 4 + 4 * n * h * dk + 4 * n, "flops": 2 * n * h * dk * dv}


def _mean_accepted(t):
    return min(2, t)   # 0 to 4, see _accept_nodes


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _parents(case, seed):
    """[n, t] int32: the parent of each drafted token, -1 for the sequence's state,
    -2 for places that hold no token.  None for full chains."""
    n, t = case["n"], case["t"]
    if case["kind"] == "chain" and not case["ragged"]:
        return None
    g = torch.Generator("cpu").manual_seed(seed + 77)
    i = torch.arange(t)
    u, w = torch.rand(n, t, generator=g), torch.rand(n, t, generator=g)
    if case["kind"] == "chain":
        par = (i - 1).expand(n, t).clone()
    elif case["kind"] == "bushy":
        # a few candidates for the first token, then siblings and continuations close by
        back = 1 + (u * 4).long()
        par = (i - back).clamp_min(-1)
    else:
        # any earlier token, or the one before
        par = torch.where(w < 0.5, i - 1, ((u * (i + 1)).long() - 1))
    if case["ragged"]:
        count = 1 + (torch.rand(n, 1, generator=g) * t).long().clamp_max(t - 1)
        par = torch.where(i < count, par, torch.full_like(par, -2))
    return par.to(torch.int32).cuda()


def _tokens(case, seed):
    """q, k (unit rows), v, beta, g of the drafted tokens and the states, as a layer has them."""
    n, t, h, dk, dv, dt = case["n"], case["t"], case["h"], case["dk"], case["dv"], DTYPES[case["dtype"]]
    g = _gen(seed)

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    q = unit(torch.randn(n, t, h, dk, generator=g, device="cuda"))
    k = unit(torch.randn(n, t, h, dk, generator=g, device="cuda"))
    v = torch.randn(n, t, h, dv, generator=g, device="cuda").to(dt)
    beta = torch.sigmoid(torch.randn(n, t, h, generator=g, device="cuda"))
    x = torch.randn(n, t, h, dk, generator=g, device="cuda")
    gate = torch.clamp(-torch.log1p(torch.exp(x)), min=-5.0)
    state = torch.randn(n, h, dk, dv, generator=g, device="cuda") * 0.2
    return dict(q=q, k=k, v=v, beta=beta, g=gate, state=state)


def _verify_inputs(case, seed):
    """Rows of a target's and a draft's probabilities that are near one another, tokens
    drawn from the draft's, and uniform random numbers in [0, 1)."""
    n, t, vocab, dt = case["n"], case["t"], case["vocab"], DTYPES[case["dtype"]]
    g = _gen(seed)
    par = _parents(case, seed)
    parents = par if par is not None else (torch.arange(t, device="cuda", dtype=torch.int32) - 1).expand(n, t)
    target = torch.empty(n, t + 1, vocab, dtype=dt, device="cuda")
    draft = torch.empty(n, t, vocab, dtype=dt, device="cuda")        # the last token has no successors
    step = max(1, (1 << 27) // ((t + 1) * vocab))
    for a in range(0, n, step):   # in parts, to bound the memory
        z = torch.randn(min(step, n - a), t + 1, vocab, generator=g, device="cuda") * 3.0
        target[a:a + step] = torch.softmax(z, -1).to(dt)
        z += 0.7 * torch.randn(z.shape, generator=g, device="cuda")
        draft[a:a + step] = torch.softmax(z[:, :t], -1).to(dt)
    rows = (parents.clamp_min(-1) + 1).long()                               # each token's context
    u = torch.rand(n, t, generator=g, device="cuda")
    tokens = torch.empty(n, t, dtype=torch.int32, device="cuda")
    for i in range(t):                                                      # drawn from the draft's rows
        c = draft[torch.arange(n, device="cuda"), rows[:, i]].float().cumsum(-1)
        tokens[:, i] = torch.searchsorted(c, (u[:, i] * c[:, -1]).unsqueeze(1)).squeeze(1).clamp_max(vocab - 1)
    uniforms = torch.rand(n, t + 1, generator=g, device="cuda")
    return dict(target=target, draft=draft if case["draft"] else None, tokens=tokens, parents=par, uniforms=uniforms)


def _accept_nodes(case, parents, seed):
    """An accepted token per sequence, at most four tokens deep (-1 for none in every ninth sequence)."""
    n, t = case["n"], case["t"]
    par = parents.cpu().long() if parents is not None else (torch.arange(t) - 1).expand(n, t)
    depth = torch.zeros(n, t + 1, dtype=torch.long)                         # column 0: the state itself
    for i in range(t):
        up = depth.gather(1, (par[:, i:i + 1] + 1).clamp_min(0)).squeeze(1)
        depth[:, i + 1] = torch.where(par[:, i] >= -1, up + 1, torch.full_like(up, -1000))
    want = torch.arange(n) % 9 % 5                                          # 0..4
    want = torch.where(torch.arange(n) % 9 == 8, torch.full_like(want, 4), want)
    fits = (depth <= want.unsqueeze(1)) & (depth >= 0)
    best = torch.where(fits, depth, torch.full_like(depth, -1)).max(1).indices - 1
    return best.to(torch.int32).cuda()


def _slots(case, seed):
    g = torch.Generator("cpu").manual_seed(seed + 5)
    return torch.randperm(case["slots"], generator=g)[:case["n"]].to(torch.int32).cuda()


def _states(case, seed, rows):
    """States as a prefill leaves them: key channels of very different sizes."""
    g = _gen(seed)
    x = torch.randn(rows, case["h"], case["dk"], case["dv"], generator=g, device="cuda")
    return x * torch.exp(1.5 * torch.randn(rows, case["h"], case["dk"], 1, generator=g, device="cuda") - 2.0)


def prepare(case, seed):
    op = case["op"]
    if op == "verify":
        s = _verify_inputs(case, seed)
    elif op in ("tree", "commit"):
        s = _tokens(case, seed)
        s["parents"] = _parents(case, seed)
        if op == "commit":
            s["accept_node"] = _accept_nodes(case, s["parents"], seed)
            s["state_out"] = torch.empty_like(s["state"])
        else:
            s["out"] = torch.empty_like(s["v"])
    else:
        dtype, _ = CACHES[case["cache"]]
        s = dict(slots=_slots(case, seed),
                 cache=torch.zeros(case["slots"], case["h"], case["dk"], case["dv"], dtype=torch.int8, device="cuda").view(dtype),
                 scales=torch.zeros(case["slots"], case["h"], case["dk"], device="cuda"))
        if op == "store":
            s["states"] = _states(case, seed, case["n"])
        else:
            for a in range(0, case["slots"], 64):
                x = _states(case, seed + a, min(64, case["slots"] - a))
                codes, scales = _quantise(x, dtype)
                s["cache"].view(torch.int8)[a:a + 64] = codes.view(torch.int8)
                s["scales"][a:a + 64] = scales
            if case["n"] > 8:
                s["slots"][::9] = -1                                        # new sequences start from zero
            s["states"] = torch.empty(case["n"], case["h"], case["dk"], case["dv"], device="cuda")
    s["op"] = op
    return s


# ---------------------------------------------------------------- the operators in plain form

def run(s):
    op = s["op"]
    if own:
        from linear_attention_08_b200 import kda
        if op == "tree":
            return kda.kda_decode_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], parents=s["parents"], out=s["out"])
        if op == "commit":
            return kda.kda_tree_commit(s["k"], s["v"], s["g"], s["beta"], s["state"], s["accept_node"], parents=s["parents"], state_out=s["state_out"])
        if op == "verify":
            return kda.kda_verify_tree(s["target"], s["tokens"], s["uniforms"], draft_probs=s["draft"], parents=s["parents"])
        if op == "store":
            return kda.kda_state_store(s["states"], s["slots"], s["cache"], s["scales"])
        return kda.kda_state_load(s["cache"], s["scales"], s["slots"], states=s["states"])
    if op == "tree":
        return _tree(s)
    if op == "commit":
        return _commit(s)
    if op == "verify":
        return _verify(s)
    if op == "store":
        return _store(s)
    return _load(s)


def _ancestors(parents, n, t):
    """anc[n, i, j]: token j lies on the path from the state to token i, i itself included;
    alive[n, i]: that path holds no empty place."""
    i = torch.arange(t, device="cuda")
    if parents is None:
        return (i.unsqueeze(1) >= i).expand(n, t, t), torch.ones(n, t, dtype=torch.bool, device="cuda")
    ok = (parents >= -1) & (parents < i)
    up = (parents.unsqueeze(2) == i) & ok.unsqueeze(2)
    anc = torch.matrix_power(torch.eye(t, device="cuda") + up, t) > 0
    alive = ~(anc & ~ok.unsqueeze(1)).any(2)
    return anc, alive


def _chunk(s, anc):
    """The tree as one chunk: per (sequence, head) the decayed keys, (I + L) and the solved
    values' right-hand side.  The log-decays' sums and the factors exp(+-sum) are held in 64 bits."""
    k, g = (s[x].transpose(1, 2).double() for x in ("k", "g"))              # [n, h, t, d]
    beta = s["beta"].transpose(1, 2).float().unsqueeze(3)
    n, h, t, _ = k.shape
    gam = anc.double().unsqueeze(1) @ g
    down, up = torch.exp(gam), k * torch.exp(-gam)
    k_in = k * down
    eye = torch.eye(t, dtype=torch.bool, device="cuda")
    strict = (anc & ~eye).unsqueeze(1)
    low = torch.where(strict, k_in @ up.transpose(2, 3), 0.0).float() * beta
    return gam, down, up, k_in.float(), low + eye, beta


def _tree(s):
    n, t = s["beta"].shape[:2]
    anc, alive = _ancestors(s["parents"], n, t)
    anc = anc & alive.unsqueeze(2) & alive.unsqueeze(1)
    gam, down, up, k_in, system, beta = _chunk(s, anc)
    q_in = s["q"].transpose(1, 2).double() * down
    pairs = torch.where(anc.unsqueeze(1), q_in @ up.transpose(2, 3), 0.0).float()
    v = s["v"].transpose(1, 2).float()
    v_new = torch.linalg.solve_triangular(system, beta * (v - k_in @ s["state"]), upper=False, unitriangular=True)
    o = q_in.float() @ s["state"] + pairs @ v_new
    o = torch.where(alive[:, None, :, None], o, 0.0)
    s["out"].copy_(o.transpose(1, 2))
    return s["out"]


def _commit(s):
    n, t = s["beta"].shape[:2]
    anc, alive = _ancestors(s["parents"], n, t)
    node = s["accept_node"].long()
    rows = torch.arange(n, device="cuda")
    taken = (node >= 0) & (node < t)
    node = node.clamp(0, t - 1)
    taken = taken & alive[rows, node]
    path = anc[rows, node] & taken.unsqueeze(1)                             # [n, t]
    anc = anc & path.unsqueeze(2) & path.unsqueeze(1)
    gam, down, up, k_in, system, beta = _chunk(s, anc)
    v = s["v"].transpose(1, 2).float()
    v_new = torch.linalg.solve_triangular(system, beta * (v - k_in @ s["state"]), upper=False, unitriangular=True)
    last = torch.where(taken[:, None, None], gam[rows, :, node], 0.0)       # [n, h, dk]
    left = torch.where(path[:, None, :, None], up * torch.exp(last).unsqueeze(2), 0.0).float()
    s["state_out"].copy_(torch.exp(last).float().unsqueeze(3) * s["state"] + left.transpose(2, 3) @ v_new)
    return s["state_out"]


def _verify(s):
    """Returns the last accepted token's place (-1: none), how many were accepted, and the
    tokens: the accepted ones, the one drawn after them, then -1."""
    target, draft, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniforms"].double()
    n, t = tokens.shape
    vocab = target.shape[2]
    rows = torch.arange(n, device="cuda")
    if s["parents"] is None:
        # a chain: every token's test at once, then the first one that fails
        at = torch.arange(t, device="cuda")
        p = target[rows.unsqueeze(1), at, tokens].double()
        q = draft[rows.unsqueeze(1), at, tokens].double() if draft is not None else torch.ones_like(p)
        ok = ((p > 0) & (u[:, :t] * q < p)).long().cumprod(1)
        count = ok.sum(1)
        node = count - 1
        failed = count < t
        rest = target[rows, count].double()
        x = tokens[rows, count.clamp_max(t - 1)]
        if draft is not None:
            less = (rest - draft[rows, count.clamp_max(t - 1)].double()).clamp_min(0.0)
        else:
            less = rest.scatter(1, x.unsqueeze(1), 0.0)
        rest = torch.where(failed.unsqueeze(1), less, rest)
        taken = ok > 0
    else:
        par = s["parents"].long()
        cur = torch.full((n,), -1, dtype=torch.long, device="cuda")
        rest = target[:, 0].double()
        total = torch.ones(n, dtype=torch.float64, device="cuda")
        taken = torch.zeros(n, t, dtype=torch.bool, device="cuda")
        for i in range(t):                                                  # in the order of the tokens
            here = (par[:, i] == cur) & (par[:, i] < i) & (par[:, i] >= -1)
            x = tokens[:, i]
            p = rest[rows, x]
            if draft is not None:
                q = draft[rows, (cur + 1).clamp_max(t - 1)].double()
                qx = q[rows, x]
                less = (rest / torch.where(total > 0, total, 1.0).unsqueeze(1) - q).clamp_min(0.0)
                left = less.sum(1)
            else:
                qx = torch.ones_like(p)
                less = rest.scatter(1, x.unsqueeze(1), 0.0)
                left = total - p
            yes = here & (p > 0) & (u[:, i] * total * qx < p)
            no = here & ~yes
            rest = torch.where(yes.unsqueeze(1), target[:, i + 1].double(), torch.where(no.unsqueeze(1), less, rest))
            total = torch.where(yes, 1.0, torch.where(no, left, total))
            cur = torch.where(yes, i, cur)
            taken[:, i] = yes
        node, count = cur, taken.sum(1)
    rest = torch.where((rest.sum(1) > 0).unsqueeze(1), rest, target[rows, node + 1].double())
    c = rest.cumsum(1)
    drawn = torch.searchsorted(c, (u[:, t] * c[:, -1]).unsqueeze(1), right=True).squeeze(1)
    last = torch.where(rest > 0, torch.arange(vocab, device="cuda"), -1).amax(1)
    drawn = torch.minimum(drawn, last)
    place = torch.arange(t + 1, device="cuda").expand(n, t + 1)
    order = torch.where(taken, place[:, :t], t).sort(1).indices             # the accepted tokens first
    out = torch.cat([tokens.gather(1, order), tokens[:, :1]], 1)
    out = torch.where(place < count.unsqueeze(1), out, torch.where(place == count.unsqueeze(1), drawn.unsqueeze(1), -1))
    return node.int(), count.int(), out.int()


def _quantise(x, dtype):
    """One scale for each row (key channel): its largest magnitude over the type's largest value."""
    top = 448.0 if dtype == torch.float8_e4m3fn else 127.0
    big = x.abs().amax(-1)
    scale = torch.where(torch.isfinite(big), big / top, math.nan)
    y = torch.where((scale > 0).unsqueeze(-1), x / scale.unsqueeze(-1), 0.0).clamp(-top, top)
    return (y.to(dtype) if dtype == torch.float8_e4m3fn else torch.round(y).to(dtype)), scale


def _store(s):
    codes, scale = _quantise(s["states"], s["cache"].dtype)
    slots = s["slots"].long()
    s["cache"].view(torch.int8)[slots] = codes.view(torch.int8)
    s["scales"][slots] = scale
    return s["cache"], s["scales"]


def _load(s):
    slots = s["slots"].long()
    at = slots.clamp_min(0)
    x = s["cache"].view(torch.int8)[at].view(s["cache"].dtype).float() * s["scales"][at].unsqueeze(-1)
    s["states"].copy_(torch.where((slots >= 0)[:, None, None, None], x, 0.0))
    return s["states"]


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None                       # whole numbers alone
    if op == "load":
        d = s["cache"].view(torch.int8)
        values = d.double() if case["cache"] == "int8" else d.view(torch.float8_e4m3fn).double()
        out = torch.zeros(s["states"].shape, dtype=torch.float64, device="cuda")
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                out[i] = values[slot] * s["scales"][slot].double()[:, :, None]
        return out
    if op == "store":
        # the codes themselves are whole values of eight bits; the scales are computed numbers
        scales = s["scales"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            scales[slot] = s["states"][i].double().abs().amax(-1) / CACHES[case["cache"]][1]
        return None, scales
    n, t, h, dk, dv = (case[x] for x in ("n", "t", "h", "dk", "dv"))
    parents = s["parents"].tolist() if s["parents"] is not None else [[i - 1 for i in range(t)]] * n
    out = torch.zeros(n, t, h, dv, dtype=torch.float64, device="cuda") if op == "tree" else s["state"].double()
    accept = s["accept_node"].tolist() if op == "commit" else None
    if op == "commit":
        # token by token along the accepted path
        for b in range(n):
            path, i = [], accept[b]
            while i >= 0:
                path.append(i)
                i = parents[b][i]
            state = out[b]
            for i in (reversed(path) if i == -1 else ()):
                state = _step(state, *(s[x][b, i].double() for x in ("k", "v", "g", "beta")))
            out[b] = state
        return out
    for a in range(0, n, 64):
        # 64 sequences at a time, node by node: each node's state from its parent's
        m = min(64, n - a)
        par = torch.tensor(parents[a:a + m], device="cuda")
        rows = torch.arange(m, device="cuda")
        for h0 in range(0, h, 8):
            hs = slice(h0, min(h, h0 + 8))
            nodes = torch.zeros(m, t + 1, len(range(h)[hs]), dk, dv, dtype=torch.float64, device="cuda")
            nodes[:, 0] = s["state"][a:a + m, hs].double()
            live = torch.zeros(m, t + 1, dtype=torch.bool, device="cuda")
            live[:, 0] = True
            for i in range(t):
                fine = (par[:, i] >= -1) & (par[:, i] < i)
                up = torch.where(fine, par[:, i] + 1, 0)
                live[:, i + 1] = fine & live[rows, up]
                x = {y: s[y][a:a + m, i, hs].double() for y in ("q", "k", "v", "g", "beta")}
                nodes[:, i + 1] = _step(nodes[rows, up], x["k"], x["v"], x["g"], x["beta"])
                o = (nodes[:, i + 1] * x["q"].unsqueeze(-1)).sum(-2)
                out[a:a + m, i, hs] = torch.where(live[:, i + 1][:, None, None], o, 0.0)
    return out


def _step(state, k, v, g, beta):
    """One token: the state decayed, then corrected towards k -> v."""
    state = torch.exp(g).unsqueeze(-1) * state
    u = beta.unsqueeze(-1) * (v - (state * k.unsqueeze(-1)).sum(-2))
    return state + k.unsqueeze(-1) * u.unsqueeze(-2)
