"""Plain references in 64 bits (numpy, token by token) of the operators of
speculative decoding and of the state cache, and inputs for their tests."""
from __future__ import annotations

import numpy as np
import torch

from linear_attention_08_b200 import inputs as kin


def f64(x):
    return x.detach().to("cpu", torch.float64).numpy() if hasattr(x, "detach") else np.asarray(x, np.float64)


def path_to(parents, node, T):
    """Places from the first drafted token to ``node``; None when it holds an empty one."""
    path, i = [], int(node)
    if not 0 <= i < T:
        return None
    while i != -1:
        up = int(parents[i]) if parents is not None else i - 1
        if up < -1 or up >= i:
            return None
        path.append(i)
        i = up
    return path[::-1]


def step(S, k, v, g, beta):
    """One token on states [H, Dk, Dv]."""
    A = np.exp(g)[:, :, None] * S
    u = beta[:, None] * (v - np.einsum("hk,hkv->hv", k, A))
    return A + k[:, :, None] * u[:, None, :]


def tree(d, parents):
    """(out, states of every place, alive) for one batch of trees."""
    q, k, v, g, beta, S0 = (f64(d[x]) for x in ("q", "k", "v", "g", "beta", "init_state"))
    N, T, H, _ = k.shape
    out = np.zeros(v.shape)
    states = np.zeros((N, T, *S0.shape[1:]))
    alive = np.zeros((N, T), dtype=bool)
    for n in range(N):
        for t in range(T):
            up = int(parents[n, t]) if parents is not None else t - 1
            if up < -1 or up >= t or (up >= 0 and not alive[n, up]):
                continue
            alive[n, t] = True
            states[n, t] = step(S0[n] if up < 0 else states[n, up], k[n, t], v[n, t], g[n, t], beta[n, t])
            out[n, t] = np.einsum("hk,hkv->hv", q[n, t], states[n, t])
    return out, states, alive


def commit(d, parents, accept):
    _, states, alive = tree(d, parents)
    S = f64(d["init_state"]).copy()
    for n, a in enumerate(np.asarray(accept)):
        if 0 <= a < states.shape[1] and alive[n, a]:
            S[n] = states[n, a]
    return S


def verify(target, draft, tokens, parents, uniforms):
    """(accept_node, accept_len, out_tokens) from the definition."""
    p, d, u = f64(target), (None if draft is None else f64(draft)), f64(uniforms)
    tok = np.asarray(tokens)
    N, T = tok.shape
    V = p.shape[2]
    node, length = np.full(N, -1), np.zeros(N, dtype=int)
    out = np.full((N, T + 1), -1)
    for n in range(N):
        par = [int(parents[n, i]) if parents is not None else i - 1 for i in range(T)]
        c, r, R = -1, p[n, 0], 1.0
        for i in range(T):
            if par[i] != c or not -1 <= par[i] < i:
                continue
            x = int(tok[n, i])
            inside = 0 <= x < V
            rx = r[x] if inside else 0.0
            dx = 1.0 if d is None else (d[n, c + 1, x] if inside else 0.0)
            if rx > 0 and u[n, i] * R * dx < rx:
                out[n, length[n]] = x
                length[n] += 1
                c, r, R = i, p[n, i + 1], 1.0
            elif d is None:
                r = r.copy()
                if inside:
                    r[x] = 0.0
                R -= rx
            else:
                r = np.maximum(r / (R if R > 0 else 1.0) - d[n, c + 1], 0.0)
                R = r.sum()
        node[n] = c
        if not r.sum() > 0:
            r = p[n, c + 1]
        if r.sum() > 0:
            C = np.cumsum(r)
            j = int(np.searchsorted(C, u[n, T] * C[-1], side="right"))
            out[n, length[n]] = min(j, int(np.nonzero(r)[0][-1]))
    return node, length, out


E4M3 = np.array([(-1) ** (b >> 7) * ((b & 7) * 2.0 ** -9 if (b >> 3) & 15 == 0
                                      else (1 + (b & 7) / 8) * 2.0 ** (((b >> 3) & 15) - 7))
                 for b in range(256)])
E4M3[[0x7F, 0xFF]] = np.nan


def quantise(states, kind):
    """(codes as values, FP32 scales) of FP32 states, one scale per row (its largest
    magnitude times 1 / top); every step rounded to FP32, codes to the nearest, ties to even."""
    x = np.asarray(states, np.float32)
    top = np.float32(448.0 if kind == "e4m3" else 127.0)
    with np.errstate(all="ignore"):
        big = np.abs(x).max(-1)
        scale = np.where(np.isfinite(x).all(-1), big * (np.float32(1) / top), np.float32(np.nan)).astype(np.float32)
        y = np.where((scale > 0)[..., None], x / scale[..., None], np.float32(0)).astype(np.float32)
    y = np.clip(y, -top, top)
    if kind == "int8":
        return np.rint(y).astype(np.float64), scale
    pos = E4M3[:0x7F]                                  # 0 .. 448, increasing; code parity = even or odd
    mag = np.abs(y).astype(np.float64)
    hi = np.searchsorted(pos, mag)                     # pos[hi - 1] < mag <= pos[hi]
    lo = np.maximum(hi - 1, 0)
    up = (pos[hi] - mag < mag - pos[lo]) | ((pos[hi] - mag == mag - pos[lo]) & (hi % 2 == 0))
    return np.where(np.signbit(y), -1.0, 1.0) * np.where(up, pos[hi], pos[lo]), scale


def make_tree(N, T, kind, seed):
    """Parents int32 [N, T] (None for "chain"): bushy, random, star, ragged, holes."""
    rng = np.random.default_rng(seed)
    i = np.arange(T)
    if kind == "chain":
        return None
    if kind == "star":
        par = np.full((N, T), -1)
    elif kind == "bushy":
        par = np.maximum(i - 1 - rng.integers(0, 4, (N, T)), -1)
    else:
        par = np.array([[rng.integers(-1, t) for t in range(T)] for _ in range(N)]).reshape(N, T)
    if kind == "ragged":
        par = np.where(i < rng.integers(0, T + 1, (N, 1)), par, -2)
    if kind == "holes":
        bad = np.array([-2, -7, 64, 2 ** 31 - 1, -2 ** 31])
        par = np.where(rng.random((N, T)) < 0.2, bad[rng.integers(0, 5, (N, T))], par)
        par[0, T - 1] = T - 1                          # its own predecessor: empty
    return torch.tensor(par, dtype=torch.int32)


def make_tokens(N, T, H, Dk, Dv, dtype, seed, state_std=0.3):
    return kin.make_inputs((N, T), H, Dk, Dv, dtype, seed, num_states=N, state_std=state_std)


def make_probs(N, T, V, dtype, seed, parents=None, spread=2.0):
    """Target and draft rows that are near one another, tokens drawn from the draft's."""
    gen = torch.Generator().manual_seed(seed)
    z = spread * torch.randn(N, T + 1, V, generator=gen)
    target = torch.softmax(z, -1)
    draft = torch.softmax(z[:, :T] + 0.7 * torch.randn(N, T, V, generator=gen), -1)
    par = parents if parents is not None else (torch.arange(T) - 1).expand(N, T)
    ctx = torch.where((par >= -1) & (par < T - 1), par + 1, 0).long()
    rows = torch.gather(draft, 1, ctx.unsqueeze(2).expand(N, T, V)) if T else draft
    tokens = torch.multinomial(rows.reshape(-1, V), 1, generator=gen).reshape(N, T).to(torch.int32)
    uniforms = torch.rand(N, T + 1, generator=gen)
    return target.to(dtype), draft.to(dtype), tokens, uniforms
