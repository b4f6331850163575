"""kda_state_store and kda_state_load: codes and scales to the bit, values to one rounding."""
import numpy as np
import pytest
import torch

import spec_ref as ref
from linear_attention_08_b200 import kda

pytestmark = pytest.mark.gpu

KINDS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def pool(num_slots, H, Dk, Dv, kind, fill=0x11):
    cache = torch.full((num_slots, H, Dk, Dv), fill, dtype=torch.int8, device="cuda").view(KINDS[kind])
    return cache, torch.full((num_slots, H, Dk), -3.0, device="cuda")


def values(cache):
    return cache.view(torch.int8).cpu().double().numpy() if cache.dtype == torch.int8 else \
        ref.E4M3[cache.view(torch.uint8).cpu().numpy()]


def make_states(n, H, Dk, Dv, seed):
    gen = torch.Generator().manual_seed(seed)
    rows = torch.exp(3 * torch.randn(n, H, Dk, 1, generator=gen))
    return torch.randn(n, H, Dk, Dv, generator=gen) * rows


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("Dk", [32, 64, 128])
@pytest.mark.parametrize("Dv", [32, 64, 128])
def test_store_and_load(kind, Dk, Dv):
    n, H, slots = 5, 3, 9
    x = make_states(n, H, Dk, Dv, seed=81)
    where = torch.tensor([7, 0, -1, 8, 9], dtype=torch.int32)     # two of them outside the cache
    cache, scales = pool(slots, H, Dk, Dv, kind)
    before = values(cache)
    kda.kda_state_store(x.cuda(), where.cuda(), cache, scales)
    codes, sc = ref.quantise(x.numpy(), kind)
    got, gs = values(cache), scales.cpu().numpy()
    for i, s in enumerate(where.tolist()):
        if 0 <= s < slots:
            np.testing.assert_array_equal(got[s], codes[i])
            np.testing.assert_array_equal(gs[s], sc[i])
    for s in (1, 2, 3, 4, 5, 6):                                  # other slots as they were
        np.testing.assert_array_equal(got[s], before[s])
        assert (gs[s] == -3).all()
    ask = torch.tensor([0, 8, -5, 7, 0, 2 ** 31 - 1], dtype=torch.int32)
    back = kda.kda_state_load(cache, scales, ask.cuda()).cpu()
    for i, (s, src) in enumerate(zip(ask.tolist(), (1, 3, None, 0, 1, None))):
        want = np.zeros((H, Dk, Dv), np.float32) if src is None else \
            codes[src].astype(np.float32) * sc[src][..., None]    # one FP32 product: the same bits
        np.testing.assert_array_equal(back[i].numpy(), want)


@pytest.mark.parametrize("kind,half", [("e4m3", 2.0 ** -4), ("int8", 0.5 / 127)])
def test_values_within_half_a_step(kind, half):
    """E4M3: half a step of the value (2^-4), or of the smallest codes (2^-10 of the scale);
    INT8: half a step of the row's scale.  Each plus the FP32 roundings of the two quotients
    and the product (3 of 2^-24)."""
    x = make_states(4, 2, 128, 128, seed=82)
    cache, scales = pool(4, 2, 128, 128, kind)
    at = torch.arange(4, dtype=torch.int32, device="cuda")
    kda.kda_state_store(x.cuda(), at, cache, scales)
    back = kda.kda_state_load(cache, scales, at).cpu().double()
    x, big = x.double(), x.double().abs().amax(-1, keepdim=True)
    if kind == "e4m3":
        bound = torch.maximum(half * x.abs(), 2.0 ** -10 * big / 448) + 3 * 2.0 ** -24 * x.abs()
    else:
        bound = half * big + 3 * 2.0 ** -24 * big
    assert ((back - x).abs() <= bound).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_odd_rows(kind):
    """Zero rows, single values, the smallest and the largest FP32 values, infinity, NaN."""
    x = torch.zeros(1, 1, 32, 32)
    x[0, 0, 1, 3] = -2.5
    x[0, 0, 2] = 1e-45
    x[0, 0, 3, ::2] = 1e-41
    x[0, 0, 4] = torch.linspace(-3.4e38, 3.4e38, 32)
    x[0, 0, 5] = torch.linspace(-1e-37, 1e-37, 32)
    x[0, 0, 6, 4] = float("inf")
    x[0, 0, 7, 9] = float("nan")
    x[0, 0, 8, 1], x[0, 0, 8, 2] = float("-inf"), float("nan")
    x[0, 0, 9] = torch.arange(32) * 0.5 - 8                       # ties of INT8 at scale 8/127 and of E4M3
    x[0, 0, 10] = torch.arange(32) - 15.0
    x[0, 0, 10, 0] = 127.0                                        # INT8 scale 1
    x[0, 0, 11] = torch.arange(32) + 0.5
    x[0, 0, 11, 0] = -127.0                                       # ties to even
    x[0, 0, 12] = 17.0 + torch.arange(32)
    x[0, 0, 12, 0] = 448.0                                        # E4M3 scale 1: ties between codes
    x[0, 0, 13] = 3.4e38 * torch.linspace(-1, 1, 32)
    cache, scales = pool(1, 1, 32, 32, kind)
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kda_state_store(x.cuda(), at, cache, scales)
    codes, sc = ref.quantise(x.numpy(), kind)
    np.testing.assert_array_equal(values(cache)[0], codes[0])
    np.testing.assert_array_equal(scales.cpu().numpy()[0], sc[0])
    back = kda.kda_state_load(cache, scales, at).cpu()[0, 0]
    assert torch.isnan(back[6:9]).all() and not back[0].any() and not back[2].any()
    # (linspace's FP32 step overflows over row 4's range, so that row is not finite either)
    fine = torch.isfinite(x[0, 0]).all(1)
    assert fine.sum() == 28 and torch.isfinite(back[fine]).all() and torch.isnan(back[~fine]).all()


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_a_slot_named_twice_keeps_the_last(kind):
    n = 700
    x = make_states(n, 2, 32, 32, seed=83)
    gen = torch.Generator().manual_seed(84)
    at = torch.randint(0, 40, (n,), generator=gen).to(torch.int32)
    codes, sc = ref.quantise(x.numpy(), kind)
    last = {int(s): i for i, s in enumerate(at)}
    for _ in range(3):
        cache, scales = pool(40, 2, 32, 32, kind)
        kda.kda_state_store(x.cuda(), at.cuda(), cache, scales)
        got, gs = values(cache), scales.cpu().numpy()
        for s, i in last.items():
            np.testing.assert_array_equal(got[s], codes[i])
            np.testing.assert_array_equal(gs[s], sc[i])


def test_large_pool_offsets():
    """Slots past 2^32 bytes of codes."""
    slots, H = 8400, 32                        # 4.4 GB of codes
    cache = torch.zeros(slots, H, 128, 128, dtype=torch.int8, device="cuda")
    scales = torch.zeros(slots, H, 128, device="cuda")
    x = make_states(2, H, 128, 128, seed=85)
    at = torch.tensor([slots - 1, 4], dtype=torch.int32, device="cuda")
    kda.kda_state_store(x.cuda(), at, cache, scales)
    codes, sc = ref.quantise(x.numpy(), "int8")
    back = kda.kda_state_load(cache, scales, at).cpu().numpy()
    np.testing.assert_array_equal(back, codes.astype(np.float32) * sc[..., None])
    used = torch.zeros(slots, dtype=torch.bool, device="cuda")
    used[at.long()] = True
    assert not scales[~used].any()


def test_cache_calls_in_a_graph():
    x = make_states(3, 2, 64, 64, seed=86).cuda()
    cache, scales = pool(4, 2, 64, 64, "e4m3")
    at = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    back = torch.empty_like(x)

    def go():
        kda.kda_state_store(x, at, cache, scales)
        kda.kda_state_load(cache, scales, at, states=back)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    x.mul_(-0.5)
    at.copy_(torch.tensor([3, 0, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = back.clone()
    go()
    torch.cuda.synchronize()
    assert torch.equal(got, back)
