"""The 8-bit state cache (gdn2_state_cache_*) against its 64-bit plain form.

Powers of two scale exactly and both formats' grids are reached by one rounding
to nearest, ties to even, so what reads back must equal the plain form."""
import numpy as np
import pytest
import torch

import gated_delta_rule_83_amd as g
from tests import operators_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def states(rng, *shape):
    S = rng.standard_normal(shape) * np.exp(3 * rng.standard_normal(shape[:-1] + (1,)))
    return torch.tensor(S.astype(np.float32), device=DEV)


def same(got, ref):
    off = np.argwhere(~((got == ref) | (np.isnan(got) & np.isnan(ref))))
    assert len(off) == 0, (len(off), tuple(off[0]), got[tuple(off[0])], ref[tuple(off[0])])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("N,P,shape", [(1, 1, (1, 16)), (3, 5, (2, 17, 32)), (6, 6, (3, 64, 64)), (9, 20, (4, 128, 128)),
                                       (2, 3, (1, 1000, 16)), (300, 301, (1, 3, 128))])
def test_round_trip(N, P, shape, fmt):
    rng = np.random.default_rng(N)
    S = states(rng, N, *shape)
    cache, scales = g.state_cache_empty(P, *shape, device=DEV)
    cache.fill_(0x3f)
    scales.fill_(127)
    before = cache.clone()
    slots = torch.tensor(rng.permutation(P)[:N].astype(np.int32), device=DEV)
    g.state_cache_store(S, slots, cache, scales, fmt=fmt)
    back = g.state_cache_load(cache, scales, slots, fmt=fmt)
    torch.cuda.synchronize()
    same(R.f64(back), R.cache_round(R.f64(S), fmt))
    others = [i for i in range(P) if i not in slots.tolist()]
    assert torch.equal(cache[others], before[others]) and (scales[others] == 127).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_grid_borders(fmt):
    """Values on, and halfway between, neighbouring codes, the largest ones, and scales at both ends."""
    top = 448.0 if fmt == "e4m3" else 127.0
    rows = []
    for e in (-126, -60, 0, 3, 90, 118):
        s = 2.0 ** e
        rows.append(np.linspace(-1, 1, 16) * top * s)          # the scale's own limit, exactly
        rows.append(np.array([top * (1 + 2.0 ** -20)] + [top / 3] * 15) * s)  # just past it: the next scale
        rows.append(np.array([top] + [k + 0.5 for k in range(15)]) * s)  # halves
        rows.append(np.array([top] + [2.0 ** -9 * k / 2 for k in range(15)]) * s)  # the smallest codes
    rows.append(np.zeros(16))
    rows.append(np.array([-0.0] * 8 + [1e-45] * 8))  # below every scale
    rows.append(np.array([3.4028234e38] + [-1e38] * 15))
    S = torch.tensor(np.array(rows, np.float32)[None], device=DEV)
    cache, scales = g.state_cache_empty(1, *S.shape[1:], device=DEV)
    slots = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.state_cache_store(S, slots, cache, scales, fmt=fmt)
    back = g.state_cache_load(cache, scales, slots, fmt=fmt)
    torch.cuda.synchronize()
    same(R.f64(back), R.cache_round(R.f64(S), fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_bad_rows_bad_slots_and_repeated_slots(fmt):
    rng = np.random.default_rng(2)
    S = states(rng, 6, 2, 20, 64)
    S[1, 0, 3, 5] = float("nan")
    S[1, 1, 4, 0] = -float("inf")
    cache, scales = g.state_cache_empty(4, 2, 20, 64, device=DEV)
    slots = torch.tensor([2, 1, -1, 2, 4, 1 << 30], dtype=torch.int32, device=DEV)
    g.state_cache_store(S, slots, cache, scales, fmt=fmt)
    ask = torch.tensor([2, 1, 0, -5, 4, 2, -(1 << 31)], dtype=torch.int32, device=DEV)
    back = R.f64(g.state_cache_load(cache, scales, ask, fmt=fmt))
    ref = R.cache_round(R.f64(S), fmt)
    assert np.array_equal(back[0], ref[3]) and np.array_equal(back[5], ref[3])  # the later of the two entries
    assert np.array_equal(back[1], ref[1], equal_nan=True) and np.isnan(back[1]).sum() == 2 * 64
    assert not back[[2, 3, 4, 6]].any()  # never written, or no slot at all


def test_many_entries_of_one_slot():
    S = torch.arange(1000, dtype=torch.float32, device=DEV)[:, None, None].expand(1000, 1, 16).contiguous()
    cache, scales = g.state_cache_empty(2, 1, 16, device=DEV)
    g.state_cache_store(S, torch.ones(1000, dtype=torch.int32, device=DEV), cache, scales, fmt="int8")
    back = g.state_cache_load(cache, scales, torch.ones(1, dtype=torch.int32, device=DEV), fmt="int8")
    same(R.f64(back[0]), R.cache_round(R.f64(S[999:]), "int8")[0])


def test_no_entries_and_a_replayed_graph():
    cache, scales = g.state_cache_empty(3, 2, 16, 32, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    g.state_cache_store(torch.empty(0, 2, 16, 32, device=DEV), none, cache, scales)
    assert g.state_cache_load(cache, scales, none).shape == (0, 2, 16, 32)
    S = states(np.random.default_rng(5), 2, 2, 16, 32)
    slots = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    out = torch.empty_like(S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.state_cache_store(S, slots, cache, scales)
        g.state_cache_load(cache, scales, slots, S=out)
    for i in range(4):
        S.copy_(states(np.random.default_rng(50 + i), 2, 2, 16, 32))
        graph.replay()
        torch.cuda.synchronize()
        same(R.f64(out), R.cache_round(R.f64(S), "e4m3"))
        assert torch.equal(g.state_cache_load(cache, scales, slots), out)


def test_offsets_past_32_bits():
    """Slots beyond byte 2^32 of the cache."""
    shape = (16, 128, 128)  # 256 KiB a state
    P = (1 << 32) // (1 << 18) + 3
    cache = torch.zeros((P,) + shape, dtype=torch.uint8, device=DEV)
    scales = torch.zeros((P,) + shape[:-1], dtype=torch.uint8, device=DEV)
    S = states(np.random.default_rng(6), 2, *shape)
    slots = torch.tensor([P - 1, 1], dtype=torch.int32, device=DEV)
    g.state_cache_store(S, slots, cache, scales)
    back = g.state_cache_load(cache, scales, slots)
    torch.cuda.synchronize()
    same(R.f64(back), R.cache_round(R.f64(S), "e4m3"))
    assert not cache[2:P - 1].any() and not cache[0].any()
