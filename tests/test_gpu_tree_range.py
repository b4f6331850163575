"""Tree decode at the ends of its range: decays at the limit of the factored products and beyond.

Bounds are per row (sequence, place, head), against m_t, the recurrence's own sums with every
term's magnitude in its place: rounding cannot cost more than a share of what was added up,
however much of it cancels.  With gates of -5 what one place adds to another's u shrinks by
e^-5 a place, so u and the output are two sums:

FP32: 64 half-steps of 2^-24 each (test_gpu_tree.py), 128 together.
BF16: operands rounded to TF32 by 0.71 units of 2^-10 at most, 2^-10.5.  An output's terms hold
four (Qt, Kh, P and u, or Qt and S0), and u's another four: 8 * 2^-10.5, and the output's own
rounding, 2^-8 of it.

With ordinary gates the magnitudes of u grow from place to place where u itself does not, and
the bounds are against s_t, the root of the sum of the squares of what is rounded: roundings
are independent, so a row of errors is of the size of one rounding times s_t.  A term of a BF16
call has up to eight of 2^-11.7 in the root mean square: 2^-10.2, taken
as 4 * 2^-10.5 = 2^-8.5; of an FP32 call 64 half-steps as above.
"""
import numpy as np
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import kda

pytestmark = pytest.mark.gpu

ROWS = ("q", "k", "v", "g", "beta")
SHAPES = [(torch.float32, (128, 128)), (torch.float32, (64, 64)), (torch.float32, (32, 128)),
          (torch.bfloat16, (128, 128)), (torch.bfloat16, (64, 64)), (torch.bfloat16, (32, 128)),
          (torch.bfloat16, (128, 64))]


def run(d, parents):
    c = {x: y.cuda() for x, y in d.items()}
    return kda.kda_decode_tree(*(c[x] for x in ROWS), c["init_state"], parents=None if parents is None else parents.cuda())


def magnitudes(d, parents):
    """m_t: the outputs with every term replaced by its magnitude, [N, T, H, Dv]."""
    q, k, v, g, beta, S0 = (ref.f64(d[x]) for x in ROWS + ("init_state",))
    q, k, v, S0 = (np.abs(x) for x in (q, k, v, S0))
    N, T, H, _ = k.shape
    out = np.zeros(v.shape)
    for n in range(N):
        us, decay = [None] * T, [None] * T
        for t in range(T):
            path = ref.path_to(parents[n] if parents is not None else None, t, T)
            if path is None:
                continue
            gam = np.cumsum(g[n, path], 0)                          # [len, H, Dk]
            kS = np.einsum("hk,hkv->hv", k[n, t] * np.exp(gam[-1]), S0[n])
            qS = np.einsum("hk,hkv->hv", q[n, t] * np.exp(gam[-1]), S0[n])
            u = v[n, t] + kS
            o = qS
            for i, s in enumerate(path[:-1]):
                w = np.exp(gam[-1] - gam[i]) * k[n, s]
                u = u + (k[n, t] * w).sum(-1)[:, None] * us[s]
                o = o + (q[n, t] * w).sum(-1)[:, None] * us[s]
            us[t] = beta[n, t][:, None] * u
            out[n, t] = o + (q[n, t] * k[n, t]).sum(-1)[:, None] * us[t]
    return out


def check_rows(out, want, m, dtype):
    err = np.linalg.norm(ref.f64(out) - want, axis=-1)
    size = np.linalg.norm(m, axis=-1)
    bound = 128 * 2.0 ** -24 * size if dtype == torch.float32 else \
        2.0 ** -8 * np.linalg.norm(want, axis=-1) + 8 * 2.0 ** -10.5 * size
    assert (err <= bound).all(), f"worst row: {np.nanmax(err / np.maximum(bound, 1e-300)):.3g} of its bound"


@pytest.mark.parametrize("dtype,dims", SHAPES)
@pytest.mark.parametrize("T,kind", [(15, "chain"), (16, "chain"), (16, "bushy")])
@pytest.mark.parametrize("scale", [1.0, 128 ** -0.5, 1e-2, 1e-5])
def test_rows_at_the_decay_limit(dtype, dims, T, kind, scale):
    """Gates of -5, the lowest there is: 16 places reach a cumulative decay of -80, and rows of
    q or k that are small must not be lost in it."""
    for small in ("q", "k"):
        d = ref.make_tokens(2, T, 2, *dims, dtype, seed=90 + T)
        d["g"] = torch.full_like(d["g"], -5.0)
        d[small] = (d[small].float() * scale).to(dtype)
        parents = ref.make_tree(2, T, kind, seed=91)
        want, _, _ = ref.tree(d, parents)
        check_rows(run(d, parents), want, magnitudes(d, parents), dtype)


@pytest.mark.parametrize("dtype,dims", SHAPES)
@pytest.mark.parametrize("T,kind", [(17, "chain"), (40, "bushy"), (64, "chain"), (64, "random")])
def test_rows_beyond_the_decay_limit(dtype, dims, T, kind):
    """Cumulative decays below -80 in every channel, in one, and resets to nothing."""
    d = ref.make_tokens(3, T, 2, *dims, dtype, seed=92 + T)
    d["g"][0] = -5.0
    d["g"][1, :, 0] = -5.0
    d["g"][1, :, 1, 7] = -5.0
    d["g"][2] = -5.0
    d["g"][2, 3, 0, 5] = -1.0e4
    parents = ref.make_tree(3, T, kind, seed=93)
    want, _, _ = ref.tree(d, parents)
    keep = np.ones(want.shape[:3], dtype=bool)
    keep[1, :, 1] = False               # (gates near zero: the bound above does not hold)
    out, m = run(d, parents), magnitudes(d, parents)
    check_rows(ref.f64(out)[keep], want[keep], m[keep], dtype)
    tol = 64 * 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8 + 8 * 2.0 ** -10.5
    a, b = ref.f64(out)[1, :, 1], want[1, :, 1]
    assert np.linalg.norm(a - b) <= tol * np.linalg.norm(b)


def spread(d, parents):
    """s_t: the root of the sum of the squares of everything that is rounded on the way to the
    outputs, [N, T, H, Dv]."""
    q, k, v, g, beta, S0 = (ref.f64(d[x]) for x in ROWS + ("init_state",))
    N, T, H, _ = k.shape
    out = np.zeros(v.shape)
    for n in range(N):
        us, ss = [None] * T, [None] * T
        for t in range(T):
            path = ref.path_to(parents[n] if parents is not None else None, t, T)
            if path is None:
                continue
            gam = np.cumsum(g[n, path], 0)
            e = np.exp(gam[-1])[:, :, None] * S0[n]
            u = v[n, t] - np.einsum("hk,hkv->hv", k[n, t], e)
            su = v[n, t] ** 2 + np.einsum("hk,hkv->hv", k[n, t] ** 2, e ** 2)
            so = np.einsum("hk,hkv->hv", q[n, t] ** 2, e ** 2)
            for i, s in enumerate(path[:-1]):
                w = np.exp(gam[-1] - gam[i]) * k[n, s]
                for x, kind in ((k[n, t] * w, "u"), (q[n, t] * w, "o")):
                    p = x.sum(-1)[:, None]
                    more = ((x ** 2).sum(-1)[:, None] + p ** 2) * us[s] ** 2 + p ** 2 * ss[s]
                    if kind == "u":
                        u, su = u - p * us[s], su + more
                    else:
                        so = so + more
            b = beta[n, t][:, None]
            us[t], ss[t] = b * u, b ** 2 * (su + u ** 2)
            x = q[n, t] * k[n, t]
            p = x.sum(-1)[:, None]
            out[n, t] = np.sqrt(so + ((x ** 2).sum(-1)[:, None] + p ** 2) * us[t] ** 2 + p ** 2 * ss[t])
    return out


@pytest.mark.parametrize("dtype,dims", SHAPES)
@pytest.mark.parametrize("T,kind", [(1, "chain"), (8, "bushy"), (16, "random"), (33, "holes"), (64, "bushy"), (64, "star")])
@pytest.mark.parametrize("gate", ["as drawn", "strong", "none"])
def test_rows_of_ordinary_trees(dtype, dims, T, kind, gate):
    """Every row by itself: one that is small or deep is not hidden behind the others."""
    d = ref.make_tokens(2, T, 2, *dims, dtype, seed=96 + T)
    if gate == "strong":
        d["g"] = torch.clamp(2.5 * d["g"], min=-5.0)
    elif gate == "none":
        d["g"] = torch.zeros_like(d["g"])
    parents = ref.make_tree(2, T, kind, seed=97)
    want, _, _ = ref.tree(d, parents)
    err = np.linalg.norm(ref.f64(run(d, parents)) - want, axis=-1)
    s = np.linalg.norm(spread(d, parents), axis=-1)
    bound = 64 * 2.0 ** -24 * s if dtype == torch.float32 else \
        2.0 ** -8 * np.linalg.norm(want, axis=-1) + 4 * 2.0 ** -10.5 * s
    assert (err <= bound).all(), f"worst row: {np.nanmax(err / np.maximum(bound, 1e-300)):.3g} of its bound"
